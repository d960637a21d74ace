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

// Four consecutive values at p (16 / 8-byte aligned).
template <int T>
__device__ __forceinline__ void load4(const void *p, float (&v)[4]) {
    if constexpr (T == QMM_F32) {
        const float4 a = __ldg(static_cast<const float4 *>(p));
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else {
        using E = typename Elem<T>::type;
        const uint2 a = __ldg(static_cast<const uint2 *>(p));
        const E *e = reinterpret_cast<const E *>(&a);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_f32(e[i]);
    }
}

__device__ __forceinline__ uint32_t codes4(const float (&v)[4], float inv) {
    const float2 a = make_float2(v[0] * inv, v[1] * inv), b = make_float2(v[2] * inv, v[3] * inv);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

struct QuantParams {
    const uint8_t *x;
    int64_t M, ldx;
    int K, kb, groups;  // groups of UNROLL blocks per row
    int64_t items;      // source rows (or output rows with a gather map) * groups
    uint8_t *q;
    int64_t ld_q;
    float *s;
    int64_t s_row, s_blk;
    const int32_t *map;
    int k;
    int64_t rows_max;
    const int32_t *count;
    unsigned *zero;
    int n_zero;
    int *status;
};

constexpr int QUANT_THREADS = 256;
constexpr int UNROLL = 4;  // blocks a warp has in flight

// One warp per group of UNROLL blocks of a row, lane i holding values
// 4i .. 4i+3 of each block.  VEC: rows, K and the base allow 4-value loads
// and 4-code stores (whole groups of four lie inside or outside the row).
template <int T, bool VEC>
__global__ void __launch_bounds__(QUANT_THREADS) f8_quantize_kernel(const QuantParams P) {
    using E = typename Elem<T>::type;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < P.n_zero; i += QUANT_THREADS) P.zero[i] = 0u;
    const int lane = threadIdx.x & 31;
    const bool gather = P.map && P.k == 0;
    int64_t rows = P.M;
    if (gather) {
        rows = P.rows_max;
        if (P.count) rows = min(rows, static_cast<int64_t>(max(__ldg(P.count), 0)));
    }
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (QUANT_THREADS / 32) + (threadIdx.x >> 5);
         it < rows * P.groups; it += static_cast<int64_t>(gridDim.x) * (QUANT_THREADS / 32)) {
        const int64_t r = it / P.groups;
        const int b0 = static_cast<int>(it - r * P.groups) * UNROLL;
        int64_t src = r;
        if (gather) {
            src = __ldg(P.map + r);
            if (src < 0 || src >= P.M) {
                if (lane == 0) atomicOr(P.status, STATUS_INDEX);
                continue;
            }
        }
        const E *row = reinterpret_cast<const E *>(P.x) + src * P.ldx;
        float v[UNROLL][4];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int c = (b0 + u) * F8_BLOCK + 4 * lane;
            if constexpr (VEC) {
                if (c < P.K) {
                    load4<T>(row + c, v[u]);
                } else {
                    v[u][0] = v[u][1] = v[u][2] = v[u][3] = 0.0f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[u][i] = c + i < P.K ? to_f32(row[c + i]) : 0.0f;
            }
        }
        uint32_t code[UNROLL];
        float scale[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) a = max(a, __float_as_uint(v[u][i]) & 0x7fffffffu);
            a = __reduce_max_sync(0xffffffffu, a);
            const float s = __fdiv_rn(__uint_as_float(a), 448.0f);
            scale[u] = s < 1.17549435e-38f ? 1.17549435e-38f : s;  // (keeps a NaN)
            code[u] = codes4(v[u], __fdiv_rn(1.0f, scale[u]));
        }
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
                const int c = (b0 + u) * F8_BLOCK + 4 * lane;
                if constexpr (VEC) {
                    if (c < P.K) *reinterpret_cast<uint32_t *>(qr + c) = code[u];
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + i < P.K) qr[c + i] = static_cast<uint8_t>(code[u] >> (8 * i));
                }
                if (lane == 0 && b0 + u < P.kb) P.s[dst * P.s_row + (b0 + u) * P.s_blk] = scale[u];
            }
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

template <int T>
cudaError_t quantize_t(const F8Quant &q, cudaStream_t st, int num_sms) {
    QuantParams p;
    p.x = static_cast<const uint8_t *>(q.x);
    p.M = q.M;
    p.ldx = q.ldx;
    p.K = static_cast<int>(q.K);
    p.kb = static_cast<int>(f8_blocks(q.K));
    p.groups = (p.kb + UNROLL - 1) / UNROLL;
    p.q = q.q;
    p.ld_q = q.ld_q;
    p.s = q.s;
    p.s_row = q.s_row;
    p.s_blk = q.s_blk;
    p.map = q.map;
    p.k = q.k;
    p.rows_max = q.rows_max;
    p.count = q.count;
    p.zero = q.zero;
    p.n_zero = q.n_zero;
    p.status = q.status;
    p.items = (q.map && q.k == 0 ? q.rows_max : q.M) * p.groups;
    const int es = f8_size(T);
    const bool vec = q.K % 4 == 0 && q.ldx % 4 == 0 && q.ld_q % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(q.x) % (4 * es) == 0 && reinterpret_cast<uintptr_t>(q.q) % 4 == 0;
    const void *kern = vec ? reinterpret_cast<const void *>(f8_quantize_kernel<T, true>)
                           : reinterpret_cast<const void *>(f8_quantize_kernel<T, false>);
    static OncePerDevice ready[2];
    const cudaError_t e = ready[vec](q.dev, [&] {
        return vec ? prefer_max_shared(f8_quantize_kernel<T, true>) : prefer_max_shared(f8_quantize_kernel<T, false>);
    });
    if (e != cudaSuccess) return e;
    const int64_t blocks = (p.items + QUANT_THREADS / 32 - 1) / (QUANT_THREADS / 32);
    const int64_t cap = static_cast<int64_t>(num_sms) * 8;
    void *args[] = {&p};
    return launch_pdl(kern, dim3(static_cast<unsigned>(blocks < 1 ? 1 : blocks < cap ? blocks : cap)),
                      dim3(QUANT_THREADS), args, st);
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
