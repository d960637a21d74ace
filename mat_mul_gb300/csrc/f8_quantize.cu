// f8_quantize.cu -- activations to e4m3 codes with one fp32 scale per 128
// values: s = max(max|x| / 448, 2^-126), q = e4m3(x * (1/s)), and the sum of
// the experts' rows.
//
// The scale, its reciprocal (IEEE divisions) and their product with x are
// each rounded to fp32, so the codes are reproducible bit for bit.  The
// maximum is taken over the bits of |x| as integers: a NaN is above infinity
// there, so a block that holds either gets a NaN or infinite scale and its
// whole product is NaN instead of silently losing the value.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "f8_internal.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qk {

namespace {

template <int T> struct Elem;
template <> struct Elem<QMM_F32> { using type = float; };
template <> struct Elem<QMM_F16> { using type = __half; };
template <> struct Elem<QMM_BF16> { using type = __nv_bfloat16; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// V consecutive values (aligned to their size, at most 16 bytes) as fp32, and
// the largest |v| as the bits of an fp32.
template <int T, int V>
__device__ __forceinline__ uint32_t load_values(const void *p, float (&v)[V]) {
    uint32_t a = 0;
    if constexpr (T == QMM_F32) {
        const float4 q = __ldg(static_cast<const float4 *>(p));
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
#pragma unroll
        for (int i = 0; i < V; ++i) a = max(a, __float_as_uint(v[i]) & 0x7fffffffu);
    } else {
        uint32_t w[V / 2];
        if constexpr (V == 8) {
            const uint4 q = __ldg(static_cast<const uint4 *>(p));
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else {
            const uint2 q = __ldg(static_cast<const uint2 *>(p));
            w[0] = q.x, w[1] = q.y;
        }
        uint32_t m = 0;  // two 16-bit maxima: |v| in either 16-bit type is in the order of its bits
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            m = __vmaxu2(m, w[i] & 0x7fff7fffu);
            if constexpr (T == QMM_BF16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
            }
        }
        m = max(m & 0xffffu, m >> 16);
        if constexpr (T == QMM_BF16) a = m << 16;
        else a = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
    }
    return a;
}

__device__ __forceinline__ uint32_t codes4(const float *v, float inv) {
    const float2 a = make_float2(v[0] * inv, v[1] * inv), b = make_float2(v[2] * inv, v[3] * inv);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

struct QuantParams {
    const uint8_t *x;
    int64_t M, ldx;
    int K, kb, groups;  // blocks of a row, and warp steps that cover them
    uint8_t *q;
    int64_t ld_q;
    float *s;
    int64_t s_row, s_blk;
    const int32_t *map;
    int k;
    int64_t rows_max;
    const int32_t *count;
    int *status;
};

constexpr int QUANT_THREADS = 256;
constexpr int UNROLL = 4;  // loads a warp has in flight

// V values per lane and load: 8 (16 lanes per block, two blocks per load; the
// 16-bit types) or 4 (the whole warp on a block).  One warp takes the
// UNROLL * 32 * V / 128 blocks of a row that UNROLL loads hold.  The two
// divisions of a block's scale are done once for all of them, by the lanes
// that each take one of the warp's blocks, instead of once per block by every
// lane: with 4 values per lane and the divisions per block the kernel was bound by
// instruction issue (8191 x 5120 bf16 39 us).  Now 24.4 us, 5.2 TB/s of the 126 MB
// it reads and writes (0.77 of the measured copy rate); 8191 x 5120 fp32 36.5 us,
// 5.8 TB/s; 4 x 4096 2.1 us, a launch and two trips to memory.
// VEC: rows, K and the bases allow whole groups of V values (inside or outside
// the row) and of V codes.
template <int T, int V, bool VEC>
__global__ void __launch_bounds__(QUANT_THREADS) f8_quantize_kernel(const QuantParams P) {
    using E = typename Elem<T>::type;
    constexpr int LPB = F8_BLOCK / V, BPL = 32 / LPB;  // lanes per block, blocks per load
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, in_block = lane % LPB;
    const bool gather = P.map && P.k == 0;
    int64_t rows = P.M;
    if (gather) {
        rows = P.rows_max;
        if (P.count) rows = min(rows, static_cast<int64_t>(max(__ldg(P.count), 0)));
    }
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (QUANT_THREADS / 32) + (threadIdx.x >> 5);
         it < rows * P.groups; it += static_cast<int64_t>(gridDim.x) * (QUANT_THREADS / 32)) {
        const int64_t r = it / P.groups;
        const int b0 = static_cast<int>(it - r * P.groups) * (UNROLL * BPL) + lane / LPB;  // this lane's first block
        int64_t src = r;
        if (gather) {
            src = __ldg(P.map + r);
            if (src < 0 || src >= P.M) {
                if (lane == 0) atomicOr(P.status, STATUS_INDEX);
                continue;
            }
        }
        const E *row = reinterpret_cast<const E *>(P.x) + src * P.ldx;
        float v[UNROLL][V];
        uint32_t a[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int c = (b0 + u * BPL) * F8_BLOCK + V * in_block;
            a[u] = 0;
            if (VEC && c < P.K) {
                a[u] = load_values<T, V>(row + c, v[u]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v[u][i] = !VEC && c + i < P.K ? to_f32(row[c + i]) : 0.0f;
                    a[u] = max(a[u], __float_as_uint(v[u][i]) & 0x7fffffffu);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if constexpr (LPB == 32) {
                a[u] = __reduce_max_sync(0xffffffffu, a[u]);
            } else {
#pragma unroll
                for (int o = LPB / 2; o > 0; o >>= 1) a[u] = max(a[u], __shfl_xor_sync(0xffffffffu, a[u], o));
            }
        }
        // lane u of a block's lanes: the maximum of load u
        static_assert(UNROLL == 4, "two selects");
        const uint32_t even = in_block & 2 ? a[2] : a[0], odd = in_block & 2 ? a[3] : a[1];
        const uint32_t mine = in_block & 1 ? odd : even;
        float scale = __fdiv_rn(__uint_as_float(mine), 448.0f);
        scale = scale < 1.17549435e-38f ? 1.17549435e-38f : scale;  // (keeps a NaN)
        const float inv_mine = __fdiv_rn(1.0f, scale);
        uint32_t code[UNROLL][V / 4];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const float inv = __shfl_sync(0xffffffffu, inv_mine, (lane & ~(LPB - 1)) + u);
#pragma unroll
            for (int i = 0; i < V / 4; ++i) code[u][i] = codes4(v[u] + 4 * i, inv);
        }
        const int sb = b0 + in_block * BPL;  // the block whose scale this lane stores
        const int copies = P.map && P.k > 0 ? P.k : 1;
        for (int j = 0; j < copies; ++j) {
            int64_t dst = r;
            if (P.map && P.k > 0) {
                dst = __ldg(P.map + r * P.k + j);
                if (dst < 0 || dst >= P.rows_max) {
                    if (lane == 0) atomicOr(P.status, STATUS_INDEX);
                    continue;
                }
            }
            uint8_t *qr = P.q + dst * P.ld_q;
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int c = (b0 + u * BPL) * F8_BLOCK + V * in_block;
                if constexpr (VEC) {
                    if (c < P.K) {
                        if constexpr (V == 8) *reinterpret_cast<uint2 *>(qr + c) = make_uint2(code[u][0], code[u][1]);
                        else *reinterpret_cast<uint32_t *>(qr + c) = code[u][0];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (c + i < P.K) qr[c + i] = static_cast<uint8_t>(code[u][i / 4] >> (8 * (i % 4)));
                }
            }
            if (in_block < UNROLL && sb < P.kb) P.s[dst * P.s_row + sb * P.s_blk] = scale;
        }
    }
}

template <int T>
__device__ __forceinline__ void store1(void *y, int64_t i, float v) {
    if constexpr (T == QMM_F32) static_cast<float *>(y)[i] = v;
    else if constexpr (T == QMM_F16) static_cast<__half *>(y)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(v);
}

struct CombineParams {
    const float *d;
    int64_t ldd, R, T, H, ldy;
    const float *w;
    const int32_t *slots;
    int k;
    void *y;
    int *status;
};

// Four columns of one token per thread and step: the k rows are added in the
// order of the token's choices, so the result does not depend on the launch.
template <int T>
__global__ void __launch_bounds__(256) f8_combine_kernel(const CombineParams P) {
    pdl_wait();
    pdl_trigger();
    const int64_t per = (P.H + 3) / 4;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; it < P.T * per;
         it += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t t = it / per, c = 4 * (it - t * per);
        float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j = 0; j < P.k; ++j) {
            const int64_t r = __ldg(P.slots + t * P.k + j);
            if (r < 0 || r >= P.R) {
                if (c == 0) atomicOr(P.status, STATUS_INDEX);
                continue;
            }
            const float w = __ldg(P.w + t * P.k + j);
            // (rows of d are 16-byte multiples, padded past H)
            const float4 v = *reinterpret_cast<const float4 *>(P.d + r * P.ldd + c);
            a[0] = fmaf(w, v.x, a[0]);
            a[1] = fmaf(w, v.y, a[1]);
            a[2] = fmaf(w, v.z, a[2]);
            a[3] = fmaf(w, v.w, a[3]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < P.H) store1<T>(P.y, t * P.ldy + c + i, a[i]);
    }
}

cudaError_t launch_pdl(const void *kern, dim3 grid, dim3 block, void **args, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

template <int T, int V, bool VEC>
cudaError_t quantize_v(const F8Quant &q, cudaStream_t st, int num_sms) {
    QuantParams p;
    p.x = static_cast<const uint8_t *>(q.x);
    p.M = q.M;
    p.ldx = q.ldx;
    p.K = static_cast<int>(q.K);
    p.kb = static_cast<int>(f8_blocks(q.K));
    constexpr int BLOCKS = UNROLL * 32 * V / F8_BLOCK;  // per warp and step
    p.groups = (p.kb + BLOCKS - 1) / BLOCKS;
    p.q = q.q;
    p.ld_q = q.ld_q;
    p.s = q.s;
    p.s_row = q.s_row;
    p.s_blk = q.s_blk;
    p.map = q.map;
    p.k = q.k;
    p.rows_max = q.rows_max;
    p.count = q.count;
    p.status = q.status;
    const int64_t items = (q.map && q.k == 0 ? q.rows_max : q.M) * p.groups;
    static OncePerDevice ready;
    const cudaError_t e = ready(q.dev, [] { return prefer_max_shared(f8_quantize_kernel<T, V, VEC>); });
    if (e != cudaSuccess) return e;
    const int64_t blocks = (items + QUANT_THREADS / 32 - 1) / (QUANT_THREADS / 32);
    const int64_t cap = static_cast<int64_t>(num_sms) * 64;
    void *args[] = {&p};
    return launch_pdl(reinterpret_cast<const void *>(f8_quantize_kernel<T, V, VEC>),
                      dim3(static_cast<unsigned>(blocks < 1 ? 1 : blocks < cap ? blocks : cap)), dim3(QUANT_THREADS), args,
                      st);
}

// 8 values per lane where 16-byte loads and 8-byte stores are aligned, else 4,
// else element by element.
template <int T>
cudaError_t quantize_t(const F8Quant &q, cudaStream_t st, int num_sms) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(q.x), c = reinterpret_cast<uintptr_t>(q.q);
    auto fits = [&](int v) {
        return q.K % v == 0 && q.ldx % v == 0 && q.ld_q % v == 0 && x % (v * f8_size(T)) == 0 && c % v == 0;
    };
    if constexpr (T != QMM_F32)
        if (fits(8)) return quantize_v<T, 8, true>(q, st, num_sms);
    return fits(4) ? quantize_v<T, 4, true>(q, st, num_sms) : quantize_v<T, 4, false>(q, st, num_sms);
}

template <int T>
cudaError_t combine_t(CombineParams &p, cudaStream_t st, int num_sms, int dev) {
    static OncePerDevice ready;
    const cudaError_t e = ready(dev, [] { return prefer_max_shared(f8_combine_kernel<T>); });
    if (e != cudaSuccess) return e;
    const int64_t blocks = (p.T * ((p.H + 3) / 4) + 255) / 256, cap = static_cast<int64_t>(num_sms) * 8;
    void *args[] = {&p};
    return launch_pdl(reinterpret_cast<const void *>(f8_combine_kernel<T>),
                      dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(256), args, st);
}

}  // namespace

cudaError_t launch_f8_quantize(const F8Quant &q, cudaStream_t st, int num_sms) {
    if (q.x_type == QMM_F32) return quantize_t<QMM_F32>(q, st, num_sms);
    if (q.x_type == QMM_F16) return quantize_t<QMM_F16>(q, st, num_sms);
    return quantize_t<QMM_BF16>(q, st, num_sms);
}

cudaError_t launch_f8_combine(const float *d, int64_t ldd, int64_t R, const float *w, const int32_t *slots, int64_t T,
                              int k, int64_t H, int y_type, void *y, int64_t ldy, int *status, cudaStream_t st,
                              int num_sms, int dev) {
    CombineParams p = {d, ldd, R, T, H, ldy, w, slots, k, y, status};
    if (y_type == QMM_F32) return combine_t<QMM_F32>(p, st, num_sms, dev);
    if (y_type == QMM_F16) return combine_t<QMM_F16>(p, st, num_sms, dev);
    return combine_t<QMM_BF16>(p, st, num_sms, dev);
}

}  // namespace qk
