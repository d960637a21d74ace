// kv_device.cuh -- device code that the rotation and the append share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv_internal.h"
#include "qmm_device.cuh"

namespace qk {

template <int T> struct KvElem;
template <> struct KvElem<QMM_F32> { using type = float; };
template <> struct KvElem<QMM_F16> { using type = __half; };
template <> struct KvElem<QMM_BF16> { using type = __nv_bfloat16; };

__device__ __forceinline__ float kv_f32(float v) { return v; }
__device__ __forceinline__ float kv_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float kv_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ void kv_put(float *p, float v) { *p = v; }
__device__ __forceinline__ void kv_put(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void kv_put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

template <int BYTES> struct Raw;
template <> struct Raw<2> { using type = uint16_t; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };

// V consecutive values, aligned to their size (V = 1: to the type's) and at
// most 16 bytes, as they are in memory, and as fp32.
template <class E, int V>
using Run = typename Raw<V * sizeof(E)>::type;
template <class E, int V>
__device__ __forceinline__ Run<E, V> load_run(const E *p) {
    return *reinterpret_cast<const Run<E, V> *>(p);
}
template <class E, int V>
__device__ __forceinline__ void values_of(const Run<E, V> &r, float *v) {
    const E *e = reinterpret_cast<const E *>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = kv_f32(e[i]);
}
template <class E, int V>
__device__ __forceinline__ void store_v(E *p, const float *v) {
    Run<E, V> r;
    E *e = reinterpret_cast<E *>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) kv_put(e + i, v[i]);
    *reinterpret_cast<Run<E, V> *>(p) = r;
}

// cos and sin of the angle that `turns` per position add up to at `pos`, times
// factor.  pos * turns mod 2^64 is the angle as a fraction of a full turn,
// exact but for the rounding of turns itself, so positions of any size keep
// the full precision of fp32 (as pos * radians in fp32 the angle of position
// 100000 would be off by up to 0.004 radians).  What is left of it after whole
// quarters, |x| <= pi/4, goes into the Taylor series: the first terms left out
// are x^11 / 11! < 1.8e-9 and x^12 / 12! < 1.2e-10.  (sincospif takes twice the
// instructions: 8191 x 40 x 128 bf16 at 36.5 us was bound by them.)
__device__ __forceinline__ float2 kv_turn(uint64_t turns, int pos, float factor) {
    const uint64_t a = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
    const uint32_t u = static_cast<uint32_t>(a >> 32), k = (u + 0x20000000u) >> 30;  // 2^32 ths of a turn, and the quarter
    const float x = static_cast<float>(static_cast<int32_t>(u - (k << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float y = x * x;
    const float s = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
    const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const float sine = k & 1 ? c : s, cosine = k & 1 ? s : c;
    return make_float2((k + 1) & 2 ? -cosine * factor : cosine * factor, k & 2 ? -sine * factor : sine * factor);
}

// A group of a head: V pairs, or 2 V values behind the turned ones.  Where its
// values lie: a run of V values at `first` and one at `second`.
template <int V>
struct Group {
    int pair;  // its first pair, or -1: not turned
    int first, second;
    bool interleaved;
    __device__ __forceinline__ Group(int g, const RopeArgs &r) {
        const int i = g * V;
        pair = 2 * i < r.rot ? i : -1;
        interleaved = r.interleaved;
        if (pair >= 0 && !interleaved) first = i, second = i + r.rot / 2;
        else first = 2 * i, second = first + V;
    }
    // values of both runs -> their turned values
    __device__ __forceinline__ void turn(float (&v)[2 * V], const float2 (&cs)[V]) const {
        if (pair < 0) return;
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float a = v[2 * i], b = v[2 * i + 1];
                v[2 * i] = a * cs[i].x - b * cs[i].y;
                v[2 * i + 1] = b * cs[i].x + a * cs[i].y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float a = v[i], b = v[V + i];
                v[i] = a * cs[i].x - b * cs[i].y;
                v[V + i] = b * cs[i].x + a * cs[i].y;
            }
        }
    }
    __device__ __forceinline__ void angles(const RopeArgs &r, int pos, float2 (&cs)[V]) const {
        if (pair < 0) return;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            cs[i] = kv_turn(__ldg(r.turns + pair + i), pos, r.factor);
            if (r.inverse) cs[i].y = -cs[i].y;
        }
    }
};

// Heads h0 .. h1 of one row, all at the angles cs: BATCH of them are read before
// any is written (y may be x), as they are in memory, so that the loads are on
// their way together and take few registers.
template <class X, class Y, int V, int BATCH>
__device__ __forceinline__ void turn_heads(const X *x, int64_t ldx, Y *y, int64_t ldy, int heads, const Group<V> &group,
                                           const float2 (&cs)[V]) {
    for (int h = 0; h < heads; h += BATCH, x += BATCH * ldx, y += BATCH * ldy) {
        Run<X, V> r[BATCH][2];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const X *p = x + min(i, heads - 1 - h) * ldx;  // (without a branch, which would part the loads)
            r[i][0] = load_run<X, V>(p + group.first);
            r[i][1] = load_run<X, V>(p + group.second);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            float v[2 * V];
            values_of<X, V>(r[i][0], v);
            values_of<X, V>(r[i][1], v + V);
            group.turn(v, cs);
            if (h + i < heads) {
                store_v<Y, V>(y + i * ldy + group.first, v);
                store_v<Y, V>(y + i * ldy + group.second, v + V);
            }
        }
    }
}

}  // namespace qk
