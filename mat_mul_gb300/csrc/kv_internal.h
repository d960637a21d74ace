// kv_internal.h -- declarations shared by the translation units of the paged
// 8-bit key and value cache: rotation, append and attention.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/qmm.h"
#include "f8_internal.h"

namespace qk {

// Least scale of a page: a page of zeros has it, and no product of a code, a
// scale and a factor near 1 leaves the normal range of fp32 because of it.
constexpr int KV_LEAST_EXP = -100;

// Rows of heads: element (t, h, i) of x at t * ld_t + h * ld_h + i.
struct Heads {
    const void *x;
    int64_t ld_t, ld_h;
    int type;
};

// Which values of a head are turned, and how (turns: 2^64 ths of a full turn
// per position of each pair).
struct RopeArgs {
    const uint64_t *turns;
    int rot;  // 0: nothing is
    int interleaved, inverse;
    float factor;
};

struct KvRope {
    Heads x, y;
    int64_t T;
    int heads, dim;
    const int32_t *positions;
    RopeArgs rope;
};
cudaError_t launch_rope(const KvRope &r, cudaStream_t st, int num_sms);

// The rows of a batch: sequence b has the rows offsets[b] .. offsets[b+1) (b ..
// b+1 where offsets is null) and lengths[b] tokens, the last of which are
// these rows; token j is in slot j % page of page table[b * ld_table + j / page].
struct KvBatch {
    const int32_t *offsets, *lengths, *table;
    int64_t ld_table;
    int width, B;
    int64_t T;
};

struct KvAppend {
    qmm_kv_cache c;
    KvBatch batch;
    Heads k, v, q, y;  // q.x null: no queries; y: the turned queries
    int q_heads;
    const int32_t *positions;  // null: a row's position in its sequence
    RopeArgs rope;
    int *status;
};
cudaError_t launch_kv_append(const KvAppend &a, cudaStream_t st, int num_sms);

struct KvAttention {
    qmm_kv_cache c;
    KvBatch batch;
    Heads q, y;
    int q_heads;
    double scale;
    int causal;
    int window;  // 0: none
    float *lse;
    char *scratch;
    unsigned *count;
    int *status;
    int dev;
    int stop;
};
// Scratch and zeroed words of a call.
struct KvPlan {
    size_t scratch;
    int64_t counters;
};
KvPlan kv_attention_plan(const KvAttention &a, int num_sms);
cudaError_t launch_kv_attention(const KvAttention &a, cudaStream_t st, int num_sms);

int f8_counters_n(const F8Context &c, cudaStream_t st, int64_t n, unsigned **ptr);  // n zeroed words

}  // namespace qk
