// f8_internal.h -- declarations shared by the translation units of the
// block-scaled 8-bit-float products: storage types, the activation
// quantiser, the (grouped) product kernel, the router and the combination of
// the experts' rows.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/qmm.h"

namespace qk {

constexpr int F8_BLOCK = 128;  // values per scale along K, rows per scale along N

inline int f8_size(int t) { return t == QMM_F32 ? 4 : 2; }
inline int64_t f8_blocks(int64_t n) { return (n + F8_BLOCK - 1) / F8_BLOCK; }

// The quantiser.  For every 128-value block b of a source row:
//   s = max(max|x| / 448, 2^-126), q = e4m3(x * (1/s)), round to nearest even.
// Rows of the output, [rows][ld_q] codes, and its scales at
// s[row * s_row + b * s_blk].  Where an output row comes from:
//   map == null            : row r from x[r], r < M;
//   map, k == 0 (gather)   : row r from x[map[r]], r < R = *count (at most
//                            rows_max), map[r] in [0, M);
//   map, k > 0  (scatter)  : x[t] goes to the rows map[t*k .. t*k+k), each in
//                            [0, rows_max), t < M.
// An index out of range raises STATUS_INDEX and its row is skipped.
struct F8Quant {
    int x_type;
    const void *x;
    int64_t M, K, ldx;
    uint8_t *q;
    int64_t ld_q;
    float *s;
    int64_t s_row, s_blk;
    const int32_t *map;
    int k;
    int64_t rows_max;
    const int32_t *count;
    int *status;
    int dev;
};
cudaError_t launch_f8_quantize(const F8Quant &q, cudaStream_t st, int num_sms);

// The product y[r, n] = sum_b xs[b, r] * Ws[e, n/128, b] * sum_{k in b} xq[r, k] * W[e, n, k]
// for the rows r of expert e, offsets[e] <= r < offsets[e+1] (offsets null:
// E = 1 and every row).  With W2 it is the gated pair: h = silu(W x) * (W2 x)
// written as 8-bit codes hq[r, n] and scales hs[n/128, r] in the quantiser's
// rounding, one block of 128 n at a time.
struct F8Gemm {
    const uint8_t *W, *W2;
    const float *Ws, *W2s;
    int E;
    int64_t N, K;
    const uint8_t *xq;
    int64_t ld_q;
    const float *xs;
    int64_t ld_s;
    const int32_t *offsets;
    int64_t R;
    int y_type;
    void *y;
    int64_t ldy;
    uint8_t *hq;
    int64_t ld_h;
    float *hs;
    int64_t ld_hs;
    float *part;      // f8_part_bytes()
    unsigned *count;  // one per CTA, zero before the launch and after it (unless a wait ran out)
    int *status;
    int dev;
    // xq null (where f8_fuses): one matrix and few rows, quantised by the product
    int x_type;
    const void *x;
    int64_t ldx;
};
bool f8_fuses(int64_t R, int64_t N, int64_t K, int num_sms);
size_t f8_part_bytes(int64_t R, int E, int64_t N, bool dual, bool grouped, int num_sms);
bool f8_available();
// The product with the tokens as TMEM lanes (f8_wide.cu), on single CTAs or, for
// one matrix, on pairs; launch_f8_gemm takes it for groups of many rows.
// cudaErrorNotSupported where the build gave it too few registers.
size_t f8_wide_part_bytes(int num_sms);
cudaError_t launch_f8_wide(const F8Gemm &g, int ctas, cudaStream_t st, int num_sms);
cudaError_t launch_f8_gemm(const F8Gemm &g, cudaStream_t st, int num_sms);

// The router (qmm_route).  hist: f8_route_hist_bytes() of scratch.
struct F8Route {
    int x_type;
    const void *x;
    int64_t T, ldx;
    int E, k, score, normalize;
    float factor;
    float *weights;
    int32_t *experts, *offsets, *rows, *slots;
    int32_t *hist;
    int dev;
};
size_t f8_route_hist_bytes(int64_t T, int E, int num_sms);
int f8_route_launches(int64_t T, int E, int num_sms);
cudaError_t launch_f8_route(const F8Route &r, cudaStream_t st, int num_sms);

// y[t] = sum_j w[t*k+j] * d[slots[t*k+j]] in j order, d [R][ldd] fp32; slots
// outside [0, R) raise STATUS_INDEX and count as zero rows.
cudaError_t launch_f8_combine(const float *d, int64_t ldd, int64_t R, const float *w, const int32_t *slots, int64_t T,
                              int k, int64_t H, int y_type, void *y, int64_t ldy, int *status, cudaStream_t st,
                              int num_sms, int dev);

// Launch attributes and what else a kernel needs once per device: `make` runs
// until it has succeeded on device `dev`.
struct OncePerDevice {
    std::atomic<uint64_t> done{0};
    template <class F>
    cudaError_t operator()(int dev, F make) {
        const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
        if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
        const cudaError_t e = make();
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// Library context for the entry points outside qmm_abi.cu.
struct F8Context {
    int dev, num_sms;
    int *status;
};
int f8_context(F8Context &c);
int f8_workspace(const F8Context &c, cudaStream_t st, size_t bytes, void **ptr);
int f8_counters(const F8Context &c, cudaStream_t st, unsigned **ptr);  // num_sms zeroed words
void clear_error();

}  // namespace qk
