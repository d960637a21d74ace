// f8_route.cu -- the router of an expert layer: the k largest logits of each
// token, their weights, and the (token, choice) pairs sorted by expert.
//
// One warp per token holds the token's logits in registers as order-preserving
// integers (index in expert order on a tie, NaN as -inf, -0 as +0) and takes
// the largest k times with two warp reductions each.  The pairs are sorted by
// counting: stable, so the rows of an expert are in token order and the
// result does not depend on the launch.  Up to FUSED tokens are one launch of
// one CTA.  More take two: the first leaves a histogram per CTA, and in the
// second each CTA adds up the histograms before its own (for many tokens and
// experts a launch in between does that once).  Bound by latency below a few
// thousand tokens and by the warp reductions above, two per choice (16384 tokens of
// 64 experts, 6 choices: 23 us, the logits at 2 % of the copy rate).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "f8_internal.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qk {

namespace {

constexpr int TOKENS = 64;  // most tokens per CTA when there are several
constexpr int FUSED = 128;  // most tokens that one CTA sorts by itself
constexpr int WARPS = 16;
constexpr int THREADS = 32 * WARPS;

struct RouteParams {
    const void *x;
    int64_t T, ldx;
    int x_type, E, k, score, normalize, fused, tokens, scanned;  // tokens per CTA; the histograms are running sums
    float factor;
    float *weights;
    int32_t *experts, *offsets, *rows, *slots, *hist;
};

__device__ __forceinline__ float load_logit(const RouteParams &P, int64_t i) {
    if (P.x_type == QMM_F32) return __ldg(static_cast<const float *>(P.x) + i);
    if (P.x_type == QMM_F16) return __half2float(static_cast<const __half *>(P.x)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(P.x)[i]);
}

// Integers in the order of the floats; 0 is below every one of them.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 + 0 = +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The choices of one token; lane j < k returns its expert.
template <int VPL>
__device__ __forceinline__ int choose(const RouteParams &P, int64_t t, int lane) {
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        float v = e < P.E ? load_logit(P, t * P.ldx + e) : 0.0f;
        if (v != v) v = -INFINITY;
        key[i] = e < P.E ? order_key(v) : 0u;
    }
    float top = 0.0f, rest = 0.0f;
    if (P.score == QMM_ROUTE_SOFTMAX) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = max(m, key[i]);
        top = key_value(__reduce_max_sync(0xffffffffu, m));
        if (top == -INFINITY) top = 0.0f;  // nothing to choose from: every weight 0
        if (!P.normalize) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (key[i]) rest += expf(key_value(key[i]) - top);
            rest = warp_sum(rest);
        }
    }
    int mine = 0;
    uint32_t mine_key = 0, first_key = 0;
    for (int j = 0; j < P.k; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = max(m, key[i]);
        m = __reduce_max_sync(0xffffffffu, m);
        unsigned at = 0xffffffffu;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
            if (key[i] == m) at = lane + 32 * i;
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (at == static_cast<unsigned>(lane + 32 * i)) key[i] = 0u;
        if (lane == j) mine = static_cast<int>(at), mine_key = m;
        if (j == 0) first_key = m;
    }
    const float v = key_value(mine_key);
    float w = 0.0f;
    if (lane < P.k) {
        if (P.score == QMM_ROUTE_SOFTMAX) {
            w = expf(v - top);
        } else if (v > 0.0f) {
            w = __fdiv_rn(1.0f, 1.0f + expf(-v));
        } else {
            // e^v / (1 + e^v).  Where all of them are tiny their quotients by the sum need not be: then all are
            // multiplied by e^-first (a token whose scores are below the smallest 64-bit float keeps weights of 0)
            const float shift = P.normalize ? fmaxf(fminf(key_value(first_key), 0.0f), -708.0f) : 0.0f;
            w = __fdiv_rn(expf(v - shift), 1.0f + expf(v));
        }
    }
    float total = P.normalize ? warp_sum(w) : P.score == QMM_ROUTE_SOFTMAX ? rest : 1.0f;
    if (total != 0.0f) w = __fdiv_rn(w, total);
    if (lane < P.k) {
        P.weights[t * P.k + lane] = w * P.factor;
        P.experts[t * P.k + lane] = mine;
    }
    return mine;
}

// Stable positions of the pairs [p0, p1) of this CTA: cnt[e] is the next row
// of expert e.  One warp, 32 pairs at a time, in order.
__device__ __forceinline__ void place(const RouteParams &P, int *cnt, const int *chosen, int64_t p0, int n, int lane) {
    for (int i = 0; i < n; i += 32) {
        const bool on = i + lane < n;
        const int e = on ? chosen[i + lane] : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (on) {
            const int row = cnt[e] + __popc(same & ((1u << lane) - 1u));
            const int64_t pair = p0 + i + lane;
            P.rows[row] = static_cast<int32_t>(pair / P.k);
            P.slots[pair] = row;
        }
        __syncwarp();
        if (on && (same >> lane) == 1u) cnt[e] += __popc(same);  // the last lane of each expert
        __syncwarp();
    }
}

// First CTA-sized scan: cnt[e] (counts) -> exclusive sums, in place; the
// total is returned.  One warp.
__device__ __forceinline__ int scan_experts(int *cnt, int E, int lane) {
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        const int v = e < E ? cnt[e] : 0;
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (e < E) cnt[e] = base + incl - v;
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return base;
}

template <int VPL>
__global__ void __launch_bounds__(THREADS) route_choose_kernel(const RouteParams P) {
    __shared__ int cnt[QMM_F8_MAX_EXPERTS];
    __shared__ int chosen[FUSED * QMM_ROUTE_MAX_K];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < P.E; e += THREADS) cnt[e] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.tokens;
    const int nt = static_cast<int>(min(static_cast<int64_t>(P.tokens), P.T - t0));
    for (int i = warp; i < nt; i += WARPS) {
        const int e = choose<VPL>(P, t0 + i, lane);
        if (lane < P.k) {
            chosen[i * P.k + lane] = e;
            atomicAdd(cnt + e, 1);
        }
    }
    __syncthreads();
    if (P.fused) {
        if (warp == 0) {
            const int total = scan_experts(cnt, P.E, lane);
            __syncwarp();
            for (int e = lane; e < P.E; e += 32) P.offsets[e] = cnt[e];
            if (lane == 0) P.offsets[P.E] = total;
            __syncwarp();
            place(P, cnt, chosen, t0 * P.k, nt * P.k, lane);
        }
    } else {
        for (int e = threadIdx.x; e < P.E; e += THREADS) P.hist[static_cast<int64_t>(blockIdx.x) * P.E + e] = cnt[e];
    }
}

// Second launch: cnt[e] = all pairs of experts before e + the pairs of e in
// CTAs before this one, then the positions.
__global__ void __launch_bounds__(THREADS) route_place_kernel(const RouteParams P) {
    __shared__ int cnt[QMM_F8_MAX_EXPERTS], before[QMM_F8_MAX_EXPERTS];
    __shared__ int chosen[TOKENS * QMM_ROUTE_MAX_K];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < P.E; e += THREADS) cnt[e] = before[e] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.tokens;
    const int n = static_cast<int>(min(static_cast<int64_t>(P.tokens), P.T - t0)) * P.k;
    for (int i = threadIdx.x; i < n; i += THREADS) chosen[i] = P.experts[t0 * P.k + i];
    if (P.scanned) {
        // the columns are summed up already: the totals follow the last CTA's row
        for (int e = threadIdx.x; e < P.E; e += THREADS) {
            cnt[e] = P.hist[static_cast<int64_t>(gridDim.x) * P.E + e];
            before[e] = P.hist[static_cast<int64_t>(blockIdx.x) * P.E + e];
        }
    } else {
        // every thread adds up one expert's column over a share of the CTAs
        const int wide = min((P.E + 31) & ~31, THREADS), shares = THREADS / wide;
        const int share = threadIdx.x / wide;
        if (share < shares)
            for (int e = threadIdx.x - share * wide; e < P.E; e += wide) {
                const int32_t *h = P.hist + e;
                int sum = 0, mine = 0;
#pragma unroll 8
                for (int b = share; b < static_cast<int>(gridDim.x); b += shares) {
                    const int v = __ldcg(h + static_cast<int64_t>(b) * P.E);
                    sum += v;
                    mine += b < static_cast<int>(blockIdx.x) ? v : 0;
                }
                atomicAdd(cnt + e, sum);
                atomicAdd(before + e, mine);
            }
    }
    __syncthreads();
    if (warp == 0) {
        const int total = scan_experts(cnt, P.E, lane);
        __syncwarp();
        if (blockIdx.x == 0) {
            for (int e = lane; e < P.E; e += 32) P.offsets[e] = cnt[e];
            if (lane == 0) P.offsets[P.E] = total;
        }
        for (int e = lane; e < P.E; e += 32) cnt[e] += before[e];
        __syncwarp();
        place(P, cnt, chosen, t0 * P.k, n, lane);
    }
}

// Between the two for many CTAs: every column of the histograms to its running
// sums, the total in the row after the last.  32 experts per CTA, 32 shares of
// the rows.
__global__ void __launch_bounds__(1024) route_scan_kernel(const RouteParams P, int rows) {
    __shared__ int part[32][33];
    const int lane = threadIdx.x & 31, share = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const int per = (rows + 31) / 32, a = min(rows, share * per), b = min(rows, a + per);
    pdl_wait();
    pdl_trigger();
    int32_t *h = P.hist + e;
    int sum = 0;
    if (e < P.E) {
#pragma unroll 8
        for (int r = a; r < b; ++r) sum += h[static_cast<int64_t>(r) * P.E];
    }
    part[share][lane] = sum;
    __syncthreads();
    int run = 0;
    for (int q = 0; q < share; ++q) run += part[q][lane];
    if (e < P.E) {
#pragma unroll 8
        for (int r = a; r < b; ++r) {
            const int v = h[static_cast<int64_t>(r) * P.E];
            h[static_cast<int64_t>(r) * P.E] = run;
            run += v;
        }
        if (share == 31) h[static_cast<int64_t>(rows) * P.E] = run;
    }
}

using Kernel = void (*)(const RouteParams);
Kernel choose_kernel(int E) {
    if (E <= 32) return route_choose_kernel<1>;
    if (E <= 64) return route_choose_kernel<2>;
    if (E <= 128) return route_choose_kernel<4>;
    if (E <= 256) return route_choose_kernel<8>;
    if (E <= 512) return route_choose_kernel<16>;
    return route_choose_kernel<32>;
}

template <class K, class... A>
cudaError_t launch(K kern, int64_t blocks, int threads, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

// One token per warp as long as that gives every SM at most one CTA, so that the
// histograms stay few, then four (1024 tokens of 128 experts: 16.5 -> 10 us with
// one).
static int tokens_per_cta(int64_t T, int num_sms) {
    return T <= FUSED ? FUSED : T <= static_cast<int64_t>(num_sms) * WARPS ? WARPS : TOKENS;
}

static int64_t ctas(int64_t T, int num_sms) {
    const int per = tokens_per_cta(T, num_sms);
    return (T + per - 1) / per;
}
// Every CTA of the second launch reads all histograms, ctas^2 * E words in all: from
// 32 MB on a launch in between sums them up once (16384 tokens of 256 experts 67 ->
// 41 us; of 64 experts, 17 MB, it took 24.7 against 22.3).
static bool scanned(int64_t T, int E, int num_sms) {
    return T > FUSED && ctas(T, num_sms) * ctas(T, num_sms) * E >= int64_t(1) << 23;
}

size_t f8_route_hist_bytes(int64_t T, int E, int num_sms) {
    return T <= FUSED ? 0 : static_cast<size_t>(ctas(T, num_sms) + 1) * E * sizeof(int32_t);
}
int f8_route_launches(int64_t T, int E, int num_sms) { return T <= FUSED ? 1 : scanned(T, E, num_sms) ? 3 : 2; }

cudaError_t launch_f8_route(const F8Route &r, cudaStream_t st, int num_sms) {
    RouteParams p = {r.x,      r.T,       r.ldx,     r.x_type,  r.E,    r.k,     r.score, r.normalize,
                     r.T <= FUSED, tokens_per_cta(r.T, num_sms), scanned(r.T, r.E, num_sms), r.factor, r.weights, r.experts, r.offsets,
                     r.rows, r.slots, r.hist};
    const int64_t blocks = ctas(r.T, num_sms);
    static OncePerDevice ready;
    cudaError_t e = ready(r.dev, [] {
        cudaError_t q = prefer_max_shared(route_place_kernel);
        if (q == cudaSuccess) q = prefer_max_shared(route_scan_kernel);
        for (int n = 32; n <= 1024 && q == cudaSuccess; n *= 2) q = prefer_max_shared(choose_kernel(n));
        return q;
    });
    if (e != cudaSuccess) return e;
    const RouteParams q = p;
    e = launch(choose_kernel(r.E), blocks, THREADS, st, q);
    if (e != cudaSuccess || p.fused) return e;
    if (p.scanned) {
        e = launch(route_scan_kernel, (r.E + 31) / 32, 1024, st, q, static_cast<int>(blocks));
        if (e != cudaSuccess) return e;
    }
    return launch(route_place_kernel, blocks, THREADS, st, q);
}

}  // namespace qk
