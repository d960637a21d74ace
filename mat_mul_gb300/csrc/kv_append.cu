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
// nothing depends on the order of blocks.
//
// Bound by memory for a prompt (every row read once, its codes written once),
// by latency for single tokens.
#include "kv_device.cuh"

namespace qk {

namespace {

struct AppendParams {
    uint8_t *codes[2];  // of keys, of values
    float *scales[2];
    int64_t pages;
    int heads, page, dim, q_heads, q_per;
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
__device__ bool find_unit(const AppendParams &P, int u, Unit &q) {
    int b = u, lo = u, n = 1, ordinal = 0;
    if (P.offsets) {
        int first = 0, last = P.B - 1;
        while (first < last) {
            const int mid = (first + last + 1) >> 1;
            if (__ldg(P.offsets + mid) / P.page + 2 * mid <= u) first = mid;
            else last = mid - 1;
        }
        b = first;
        lo = __ldg(P.offsets + b);
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
    if (q.page < 0 || q.page >= P.pages) {
        atomicOr(P.status, STATUS_INDEX);
        return false;
    }
    q.row = lo + (p0 - start);
    q.pos = static_cast<int>(p0);
    q.n = static_cast<int>(p1 - p0);
    return true;
}

// An infinity has no code: it becomes a NaN.
__device__ __forceinline__ float scaled(float v, float inv) {
    return fabsf(v) <= 3.402823466e38f ? v * inv : __uint_as_float(0x7fffffffu);
}
__device__ __forceinline__ uint32_t codes2(float a, float b, float inv) {
    return __nv_cvt_float2_to_fp8x2(make_float2(scaled(a, inv), scaled(b, inv)), __NV_SATFINITE, __NV_E4M3);
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
template <int T, int V, int THREADS, int KEEP>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(const AppendParams P) {
    using X = typename KvElem<T>::type;
    __shared__ float reduced[THREADS / 32 + 1];
    pdl_wait();
    pdl_trigger();
    Unit u;
    if (!find_unit(P, blockIdx.x, u)) return;
    const int groups = P.dim / (2 * V), items = u.n * groups;
    const int tid = threadIdx.x, part = blockIdx.y;
    if (part >= 2 * P.heads) {  // queries
        constexpr int BATCH = 2;
        const int h0 = (part - 2 * P.heads) * P.q_per, h1 = min(P.q_heads, h0 + P.q_per);
        for (int i = tid; i < items; i += THREADS) {
            const int t = i / groups;
            const Group<V> group(i - t * groups, P.rope);
            const int64_t row = u.row + t;
            float2 cs[V];
            group.angles(P.rope, P.positions ? __ldg(P.positions + row) : u.pos + t, cs);
            const X *x = static_cast<const X *>(P.x[2]) + row * P.ld_t[2] + h0 * P.ld_h[2];
            X *y = static_cast<X *>(P.y) + row * P.ldy_t + h0 * P.ldy_h;
            for (int h = h0; h < h1; h += BATCH, x += BATCH * P.ld_h[2], y += BATCH * P.ldy_h) {
                float v[BATCH][2 * V];
#pragma unroll
                for (int j = 0; j < BATCH; ++j)
                    if (h + j < h1) {
                        load_v<X, V>(x + j * P.ld_h[2] + group.first, v[j]);
                        load_v<X, V>(x + j * P.ld_h[2] + group.second, v[j] + V);
                    }
#pragma unroll
                for (int j = 0; j < BATCH; ++j)
                    if (h + j < h1) {
                        group.turn(v[j], cs);
                        store_v<X, V>(y + j * P.ldy_h + group.first, v[j]);
                        store_v<X, V>(y + j * P.ldy_h + group.second, v[j] + V);
                    }
            }
        }
        return;
    }
    const int is_v = part >= P.heads, head = part - is_v * P.heads;
    RopeArgs rope = P.rope;
    if (is_v) rope.rot = 0;
    const X *x = static_cast<const X *>(P.x[is_v]) + u.row * P.ld_t[is_v] + head * P.ld_h[is_v];
    const int64_t slot = u.pos % P.page, tile = static_cast<int64_t>(u.page) * P.heads + head;
    uint8_t *codes = P.codes[is_v] + tile * P.page * P.dim;
    float *scale = P.scales[is_v] + tile;
    const float before = slot ? *scale : 0.0f;

    auto values = [&](int i, float (&v)[2 * V]) {
        const int t = i / groups;
        const Group<V> group(i - t * groups, rope);
        const X *p = x + t * P.ld_t[is_v];
        load_v<X, V>(p + group.first, v);
        load_v<X, V>(p + group.second, v + V);
        if (group.pair >= 0) {
            float2 cs[V];
            group.angles(rope, P.positions ? __ldg(P.positions + u.row + t) : u.pos + t, cs);
            group.turn(v, cs);
        }
    };
    auto largest = [](float a, const float (&v)[2 * V]) {
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) {
            const float m = fabsf(v[j]);
            a = m <= 3.402823466e38f ? fmaxf(a, m) : a;  // of the finite ones
        }
        return a;
    };
    float v[KEEP ? KEEP : 1][2 * V];
    float top = 0.0f;
    if constexpr (KEEP > 0) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k) {
            const int i = tid + k * THREADS;
            if (i < items) {
                values(i, v[k]);
                top = largest(top, v[k]);
            }
        }
    } else {
        for (int i = tid; i < items; i += THREADS) {
            values(i, v[0]);
            top = largest(top, v[0]);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if constexpr (THREADS > 32) {
        if ((tid & 31) == 0) reduced[tid >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, reduced[w]);
    }
    // the smallest power of two with top <= 1.75 * 2^8 of it: one more where
    // the mantissa of top is above 1.75
    const int e = max(static_cast<int>((__float_as_uint(top) + 0x1fffffu) >> 23) - 127 - 8, KV_LEAST_EXP);
    const float s = fmaxf(pow2f(e), before), inv = __fdiv_rn(1.0f, s);
    if (slot && s != before) {
        const float ratio = before * inv;
        uint4 *w = reinterpret_cast<uint4 *>(codes);
        for (int i = tid; i < static_cast<int>(slot) * P.dim / 16; i += THREADS) {
            const uint4 q = w[i];
            w[i] = make_uint4(rescale4(q.x, ratio), rescale4(q.y, ratio), rescale4(q.z, ratio), rescale4(q.w, ratio));
        }
    }
    // (every thread has read the old scale above, before the barrier of the maximum)
    if (THREADS == 32) __syncwarp();
    if (tid == 0 && s != before) *scale = s;
    codes += slot * P.dim;
    auto put = [&](int i, const float (&w)[2 * V]) {
        const int t = i / groups;
        const Group<V> group(i - t * groups, rope);
        store_codes<V>(codes + t * P.dim + group.first, w, inv);
        store_codes<V>(codes + t * P.dim + group.second, w + V, inv);
    };
    if constexpr (KEEP > 0) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (tid + k * THREADS < items) put(tid + k * THREADS, v[k]);
    } else {
        for (int i = tid; i < items; i += THREADS) {
            values(i, v[0]);
            put(i, v[0]);
        }
    }
}

template <int T, int V, int THREADS, int KEEP>
cudaError_t launch_one(const AppendParams &p, unsigned units, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units, static_cast<unsigned>(2 * p.heads + (p.q_heads ? (p.q_heads + p.q_per - 1) / p.q_per : 0)));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<T, V, THREADS, KEEP>, p);
}

template <int T>
cudaError_t launch_t(const AppendParams &p, bool wide, unsigned units, cudaStream_t st) {
    if (!p.offsets) return wide ? launch_one<T, 4, 32, 1>(p, units, st) : launch_one<T, 1, 32, 0>(p, units, st);
    if (!wide) return launch_one<T, 1, 256, 0>(p, units, st);
    const int values = p.page * p.dim;  // of a block: KEEP groups of 8 per thread hold them
    if (values <= 8192) return launch_one<T, 4, 256, 4>(p, units, st);
    if (values <= 16384) return launch_one<T, 4, 256, 8>(p, units, st);
    return launch_one<T, 4, 512, 8>(p, units, st);
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
    bool wide = a.rope.rot % 8 == 0;
    auto runs_of_4 = [&](const Heads &h, int heads) {
        const int es = f8_size(h.type);
        return reinterpret_cast<uintptr_t>(h.x) % (4 * es) == 0 && (T == 1 || h.ld_t % 4 == 0) && (heads == 1 || h.ld_h % 4 == 0);
    };
    p.q_heads = a.q.x ? a.q_heads : 0;
    for (int i = 0; i < 3; ++i) {
        p.x[i] = in[i]->x, p.ld_t[i] = in[i]->ld_t, p.ld_h[i] = in[i]->ld_h;
        if (in[i]->x) wide = wide && runs_of_4(*in[i], i == 2 ? a.q_heads : p.heads);
    }
    if (a.q.x) wide = wide && runs_of_4(a.y, a.q_heads);
    p.y = const_cast<void *>(a.y.x), p.ldy_t = a.y.ld_t, p.ldy_h = a.y.ld_h;
    p.offsets = a.batch.offsets, p.lengths = a.batch.lengths, p.table = a.batch.table, p.positions = a.positions;
    p.ld_table = a.batch.ld_table, p.T = T, p.width = a.batch.width, p.B = a.batch.B;
    p.rope = a.rope;
    p.status = a.status;
    p.q_per = a.batch.offsets ? 8 : 2;
    const int64_t units = a.batch.offsets ? T / p.page + 2 * int64_t(p.B) : p.B;
    if (units > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const unsigned n = static_cast<unsigned>(units);
    if (a.k.type == QMM_F32) return launch_t<QMM_F32>(p, wide, n, st);
    if (a.k.type == QMM_F16) return launch_t<QMM_F16>(p, wide, n, st);
    return launch_t<QMM_BF16>(p, wide, n, st);
}

}  // namespace qk
