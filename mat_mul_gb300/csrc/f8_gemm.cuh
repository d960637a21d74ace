// f8_gemm.cuh -- what the two block-scaled 8-bit-float product kernels share:
// TMA and tcgen05 wrappers, and the count of the tiles of every expert.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "f8_internal.h"
#include "f8_schedule.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qk {
namespace f8 {

constexpr int BK = 128;        // values of K per stage: one scale block

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// Bring a box into L2.
__device__ __forceinline__ void prefetch_2d(const CUtensorMap *map, int c0, int c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1)
                 : "memory");
}

// One lane of a converged warp, the same one each time.  The compiler knows
// that a branch on it holds one thread, and feeds the tensor-core and copy
// instructions their uniform registers directly: behind "lane == 0" four MMAs
// and two commits took 745 cycles to issue, behind this 410 (a K block of
// 128 x 256 takes the tensor cores 512).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// mbar_wait without the long sleep: the stages of these kernels change hands
// every few hundred cycles.
__device__ __forceinline__ bool mbar_spin(uint32_t bar, uint32_t parity, int *status) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (clock64() - t0 > WAIT_LIMIT_CYCLES) {
            atomicOr(status, STATUS_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ void copy4(uint32_t dst, const float *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// K-major operand in 128-byte swizzled rows, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr) {
    uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// N consecutive fp32 columns of this warp's 32 TMEM lanes: issue, then wait.
// The wait takes the registers as operands so that no use of them moves
// before it.
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a));
}
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// silu(g) = g / (1 + e^-g), for g < 0 as g e^g / (1 + e^g): the exponential is
// at most 1, so nothing overflows where the result does not vanish, and the
// hardware's division has a divisor between 1 and 2.  Over all floats (each one
// tried against 64 bits) the result is within 5.3 * 2^-24 of its value, an IEEE
// division 4.8; below -87.3, where e^g is subnormal, within |g| 2^-150.  With
// __expf it was off by up to 9 * 2^-24 at -8 and 66 at -87, and 0 below.  A layer
// of 4093 tokens and 32 experts of 2048 x 1408: 239 us, with the IEEE division 252,
// with __expf 233.
__device__ __forceinline__ float silu(float g) {
    const float e = expf(-fabsf(g));
    return __fdividef(g < 0.0f ? g * e : g, 1.0f + e);
}

// Tiles before each expert, cum[0 .. E], for tiles of `tokens` rows times nb
// row blocks of W; one warp.  Groups that group_tiles() does not take raise
// STATUS_INDEX and leave their expert without tiles.
__device__ __forceinline__ void count_tiles(int *cum, const int32_t *offsets, int E, int R, int tokens, int nb, int lane,
                                            int *status) {
    int base = 0, highest = 0;
    bool fallen = false;  // an offset below the one before it
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        const int lo = offsets && e < E ? __ldg(offsets + e) : 0;
        const int hi = e >= E ? 0 : offsets ? __ldg(offsets + e + 1) : R;
        int top = lo;  // the largest of offsets[0 .. e]: the last, as long as they rise
        fallen = fallen || __any_sync(0xffffffffu, e < E && hi < lo);
        if (fallen) {
            top = max(lo, highest);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, top, o);
                if (lane >= o) top = max(top, v);
            }
            highest = __shfl_sync(0xffffffffu, top, 31);
        }
        int t = 0;
        if (e < E) {
            t = group_tiles(lo, hi, top, R, tokens, nb);
            if (t < 0) {
                atomicOr(status, STATUS_INDEX);
                t = 0;
            }
        }
        int incl = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (e < E) cum[e] = base + incl - t;
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) cum[E] = base;
}

// Rows of codes [rows][K], ld bytes apart, in boxes of 128 bytes x box_rows.
inline bool encode_rows(CUtensorMap *m, const void *base, int64_t rows, int64_t K, int64_t ld, int box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
    const cuuint32_t box[2] = {BK, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t es[2] = {1, 1};
    return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace f8
}  // namespace qk
