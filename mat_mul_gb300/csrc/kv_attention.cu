// kv_attention.cu -- which attention kernel takes a call, and what it needs.
#include "kv_attention.cuh"

namespace qk {

namespace {

// Query rows per block of the kernel for few rows: what the sequences have on
// the average, so that a decode step does not compute empty rows.
int row_groups(const KvAttention &a) {
    const int64_t rows = a.batch.T * (a.q_heads / a.c.heads) / a.batch.B;
    return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}

// Whether the call's rows go to a kernel for many rows (of 256 on tcgen05 for 16-bit
// queries, of 128 on mma.sync for fp32): heads of up to 128 values, sequences of more than 32
// rows per cache head on the average.  Measured, a kernel for few rows against the
// other, 8 sequences, 8 heads of 128: fp16, 20 rows over 1024, 4096, 16384 tokens 23, 41, 95
// against 31, 47, 125 us; fp32, 40 rows over 4096 98 against 78, 64 rows over 1024 47
// against 43.
bool many_rows(const KvAttention &a) {
    return a.c.dim <= 128 && a.batch.T * (a.q_heads / a.c.heads) > 32 * int64_t(a.batch.B);
}

// Whether few rows go to the kernel whose warps each take all rows of their tokens:
// 16-bit queries, heads of up to 128 values, 9 to 32 rows, and sequences that may be
// long (the lengths are on the device; the table says how long at most): eight tiles
// of 128 tokens per multiprocessor.  Its blocks start and end 3 us later, its tiles take
// 0.6 of the time.  Measured, the other kernel against it, 8 sequences, 8 heads of 128: 20 fp16 rows
// over 1024, 4096, 16384 tokens 22.9, 46, 120 against 26.8, 41, 95 us, 12 rows over 1024,
// 4096 16.5, 30.8 against 20.6, 28.8; 4 rows, 64 sequences of 4096 tokens, 94 against 109.
bool slim_rows(const KvAttention &a, int num_sms) {
    const double tiles = double(a.batch.width) * a.c.page / kv::TILE * a.batch.B * a.c.heads;
    return a.q.type != QMM_F32 && a.c.dim <= 128 && row_groups(a) > 1 && tiles >= 8.0 * num_sms;
}

int padded_dim(const KvAttention &a) { return a.c.dim <= 64 ? 64 : a.c.dim <= 128 ? 128 : 256; }

}  // namespace

KvPlan kv_attention_plan(const KvAttention &a, int num_sms) {
    const int64_t blocks = num_sms * 2, floats = 8 * row_groups(a) * (padded_dim(a) + 2);
    size_t bytes = static_cast<size_t>(blocks * 2 * floats * 4);
    if (many_rows(a)) {
        const int dim = static_cast<int>(a.c.dim);
        const size_t many = a.q.type == QMM_F32 ? kv::rows_part_bytes(dim, num_sms) : kv::tc_part_bytes(dim, num_sms);
        bytes = many > bytes ? many : bytes;
    }
    return {bytes, blocks};
}

cudaError_t launch_kv_attention(const KvAttention &a, cudaStream_t st, int num_sms) {
    kv::AttnParams p = {};
    p.codes[0] = static_cast<const uint8_t *>(a.c.k), p.codes[1] = static_cast<const uint8_t *>(a.c.v);
    p.scales[0] = a.c.k_scale, p.scales[1] = a.c.v_scale;
    p.pages = a.c.pages;
    p.heads = static_cast<int>(a.c.heads), p.page = static_cast<int>(a.c.page), p.dim = static_cast<int>(a.c.dim);
    p.group = a.q_heads / p.heads;
    p.q = a.q.x, p.ldq_t = a.q.ld_t, p.ldq_h = a.q.ld_h, p.q_type = a.q.type;
    p.y = const_cast<void *>(a.y.x), p.ldy_t = a.y.ld_t, p.ldy_h = a.y.ld_h, p.y_type = a.y.type;
    p.offsets = a.batch.offsets, p.lengths = a.batch.lengths, p.table = a.batch.table;
    p.ld_table = a.batch.ld_table, p.T = a.batch.T, p.width = a.batch.width, p.B = a.batch.B;
    const double factor = a.scale * 1.4426950408889634074;
    p.factor = static_cast<float>(factor);
    p.factor_low = static_cast<float>(factor - p.factor);
    p.causal = a.causal, p.window = a.window;
    for (p.div_shift = 31; (int64_t(1) << (p.div_shift - 31)) < p.group;) ++p.div_shift;
    p.div_mul = static_cast<uint32_t>(((uint64_t(1) << p.div_shift) + p.group - 1) / p.group);
    p.lse = a.lse;
    p.part = reinterpret_cast<float *>(a.scratch);
    p.count = a.count;
    p.status = a.status;
    p.stop = a.stop;
    if (many_rows(a)) {
        const cudaError_t e = a.q.type == QMM_F32 ? kv::launch_rows(p, st, num_sms, a.dev) : kv::launch_tc(p, st, num_sms, a.dev);
        if (e != cudaErrorNotSupported) return e;  // (else the build gave it too few registers)
    }
    if (slim_rows(a, num_sms)) {
        const cudaError_t e = kv::launch_slim(p, 8 * row_groups(a), st, num_sms, a.dev);
        if (e != cudaErrorNotSupported) return e;
    }
    const int nb = row_groups(a);
    const bool hl = a.q.type == QMM_F32;
    switch (padded_dim(a)) {
    case 64: return kv::launch_few_64(p, nb, hl, st, num_sms, a.dev);
    case 128: return kv::launch_few_128(p, nb, hl, st, num_sms, a.dev);
    default: return kv::launch_few_256(p, nb, hl, st, num_sms, a.dev);
    }
}

}  // namespace qk
