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
// most 16 bytes.
template <class E, int V>
__device__ __forceinline__ void load_v(const E *p, float *v) {
    using R = typename Raw<V * sizeof(E)>::type;
    const R r = *reinterpret_cast<const R *>(p);
    const E *e = reinterpret_cast<const E *>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = kv_f32(e[i]);
}
template <class E, int V>
__device__ __forceinline__ void store_v(E *p, const float *v) {
    using R = typename Raw<V * sizeof(E)>::type;
    R r;
    E *e = reinterpret_cast<E *>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) kv_put(e + i, v[i]);
    *reinterpret_cast<R *>(p) = r;
}

// cos and sin of the angle that `turns` per position add up to at `pos`, times
// factor.  pos * turns mod 2^64 is the angle as a fraction of a full turn,
// exact but for the rounding of turns itself, so positions of any size keep
// the full precision of fp32 (as pos * radians in fp32 the angle of position
// 100000 would be off by up to 0.004 radians).
__device__ __forceinline__ float2 kv_turn(uint64_t turns, int pos, float factor) {
    const uint64_t a = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
    const float half_turns = static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * factor, s * factor);
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

}  // namespace qk
