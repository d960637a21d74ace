// f8_abi.cu -- C entry points of the block-scaled 8-bit-float products and of
// the expert layer: argument checks, workspace layout and launch order.
#include <cuda_runtime.h>

#include "abi_checks.h"

namespace {

int check_rows(const void *p, int type, int64_t rows, int64_t cols, int64_t ld, const char *what) {
    if (rows > 1 && ld < cols)
        return refuse(QMM_EINVAL_SHAPE, "%s: a row pitch of %lld is less than the %lld values of a row", what,
                      static_cast<ll>(ld), static_cast<ll>(cols));
    if (!p) return refuse(QMM_EINVAL_PTR, "%s is null", what);
    if (!aligned(p, qk::f8_size(type)))
        return refuse(QMM_EINVAL_PTR, "%s must be aligned to its values (%d bytes)", what, qk::f8_size(type));
    return QMM_OK;
}
int check_matrix(const void *W, const float *S, const char *what) {
    if (!W || !S) return refuse(QMM_EINVAL_PTR, "%s: codes or scales are null", what);
    if (!aligned(W, 16)) return refuse(QMM_EINVAL_PTR, "%s: codes must be 16-byte aligned", what);
    if (!aligned(S, 4)) return refuse(QMM_EINVAL_PTR, "%s: scales must be 4-byte aligned", what);
    return QMM_OK;
}
// Sizes of a (grouped) product: what the kernel's 32-bit coordinates hold.
int check_sizes(int64_t E, int64_t N, int64_t K, int64_t R) {
    if (N < 0 || K < 0 || R < 0 || K % 16 || K > (int64_t(1) << 24))
        return refuse(QMM_EINVAL_SHAPE, "N=%lld K=%lld rows=%lld: sizes must be >= 0, K a multiple of 16 up to 2^24",
                      static_cast<ll>(N), static_cast<ll>(K), static_cast<ll>(R));
    // one bound at a time, so that no product can wrap
    if (N >= I31 || R >= I31 - 256 || E * N >= I31 - 256 || (R / 16 + E) * qk::f8_blocks(N) >= I31)
        return refuse(QMM_EINVAL_SHAPE, "E=%lld N=%lld rows=%lld: too large", static_cast<ll>(E), static_cast<ll>(N),
                      static_cast<ll>(R));
    return QMM_OK;
}
int check_experts(int64_t E) {
    if (E < 1 || E > QMM_F8_MAX_EXPERTS)
        return refuse(QMM_EINVAL_SHAPE, "E=%lld: 1 to %d experts", static_cast<ll>(E), QMM_F8_MAX_EXPERTS);
    return QMM_OK;
}

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

int zero_rows(void *y, int type, int64_t rows, int64_t cols, int64_t ldy, cudaStream_t st) {
    const size_t es = qk::f8_size(type);
    const cudaError_t e = cudaMemset2DAsync(y, static_cast<size_t>(rows > 1 ? ldy : cols) * es, 0,
                                            static_cast<size_t>(cols) * es, static_cast<size_t>(rows), st);
    return e == cudaSuccess ? QMM_OK : cuda_error(e, "zero fill");
}

// Quantised rows in the workspace: codes [rows][ld] and scales [K/128][ld_s].
struct Codes {
    int64_t ld, ld_s;
    size_t q_bytes, s_bytes;
    Codes(int64_t rows, int64_t K)
        : ld(up(K, 16)), ld_s(up(rows, 4)), q_bytes(static_cast<size_t>(up(rows * ld, 1024))),
          s_bytes(static_cast<size_t>(up(qk::f8_blocks(K) * ld_s * 4, 1024))) {}
};

// The product of one matrix (offsets null) or of E matrices over row groups.
int product(const void *W, const float *S, int64_t E, int64_t N, int64_t K, int x_type, const void *x, int64_t M,
            int64_t ldx, const int32_t *offsets, const int32_t *rows, int64_t R, int y_type, void *y, int64_t ldy,
            cudaStream_t st) {
    qk::F8Context c;
    if (int rc = qk::f8_context(c)) return rc;
    if (!qk::f8_available()) return refuse(QMM_ECUDA, "the driver has no tensor map encoder");
    const qk::CallLock lock(c.dev, st);
    // workspace: codes and scales of x (unless the product quantises x itself) |
    // partial tiles
    const bool fuse = !offsets && qk::f8_fuses(R, N, K, c.num_sms);
    const Codes q(fuse ? 0 : R, K);
    char *ws = nullptr;
    const size_t part = qk::f8_part_bytes(R, static_cast<int>(E), N, false, offsets != nullptr, c.num_sms);
    if (int rc = qk::f8_workspace(c, st, q.q_bytes + q.s_bytes + part, reinterpret_cast<void **>(&ws))) return rc;
    qk::F8Gemm g = {};
    if (int rc = qk::f8_counters(c, st, &g.count)) return rc;
    if (fuse) {
        g.x_type = x_type;
        g.x = x;
        g.ldx = ldx;
    } else {
        qk::F8Quant f = {};
        f.x_type = x_type;
        f.x = x;
        f.M = M;
        f.K = K;
        f.ldx = ldx;
        f.q = reinterpret_cast<uint8_t *>(ws);
        f.ld_q = q.ld;
        f.s = reinterpret_cast<float *>(ws + q.q_bytes);
        f.s_row = 1;
        f.s_blk = q.ld_s;
        f.map = rows;
        f.rows_max = R;
        f.count = rows ? offsets + E : nullptr;
        f.status = c.status;
        f.dev = c.dev;
        const cudaError_t e = qk::launch_f8_quantize(f, st, c.num_sms);
        if (e != cudaSuccess) return cuda_error(e, "quantize launch");
        qk::count_launches(1);
        g.xq = f.q;
        g.ld_q = q.ld;
        g.xs = f.s;
        g.ld_s = q.ld_s;
    }
    g.W = static_cast<const uint8_t *>(W);
    g.Ws = S;
    g.E = static_cast<int>(E);
    g.N = N;
    g.K = K;
    g.offsets = offsets;
    g.R = R;
    g.y_type = y_type;
    g.y = y;
    g.ldy = ldy;
    g.part = reinterpret_cast<float *>(ws + q.q_bytes + q.s_bytes);
    g.status = c.status;
    g.dev = c.dev;
    const cudaError_t e = qk::launch_f8_gemm(g, st, c.num_sms);
    if (e != cudaSuccess) return cuda_error(e, "product launch");
    qk::count_launches(1);
    return QMM_OK;
}

}  // namespace

extern "C" {

int qmm_f8_quantize(int x_type, const void *x, int64_t M, int64_t K, int64_t ldx, void *q, float *s, void *stream) {
    qk::clear_error();
    if (int rc = check_ftype(x_type, "x")) return rc;
    if (M < 0 || K < 0 || K > (int64_t(1) << 30) || M >= I31)
        return refuse(QMM_EINVAL_SHAPE, "M=%lld K=%lld: 0 <= M < 2^31, 0 <= K <= 2^30", static_cast<ll>(M), static_cast<ll>(K));
    if (M == 0 || K == 0) return QMM_OK;
    if (int rc = check_rows(x, x_type, M, K, ldx, "x")) return rc;
    if (!q) return refuse(QMM_EINVAL_PTR, "q is null");
    if (int rc = check_words(s, "s")) return rc;
    qk::F8Context c;
    if (int rc = qk::f8_context(c)) return rc;
    qk::F8Quant f = {};
    f.x_type = x_type;
    f.x = x;
    f.M = M;
    f.K = K;
    f.ldx = M > 1 ? ldx : K;
    f.q = static_cast<uint8_t *>(q);
    f.ld_q = K;
    f.s = s;
    f.s_row = qk::f8_blocks(K);
    f.s_blk = 1;
    f.status = c.status;
    f.dev = c.dev;
    const cudaError_t e = qk::launch_f8_quantize(f, static_cast<cudaStream_t>(stream), c.num_sms);
    if (e != cudaSuccess) return cuda_error(e, "quantize launch");
    qk::count_launches(1);
    return QMM_OK;
}

int qmm_f8(const void *W, const float *S, int64_t N, int64_t K, int x_type, const void *x, int64_t M, int64_t ldx,
           int y_type, void *y, int64_t ldy, void *stream) {
    qk::clear_error();
    if (int rc = check_ftype(x_type, "x")) return rc;
    if (int rc = check_ftype(y_type, "y")) return rc;
    if (int rc = check_sizes(1, N, K, M)) return rc;
    if (M == 0 || N == 0) return QMM_OK;
    if (int rc = check_rows(y, y_type, M, N, ldy, "y")) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) return zero_rows(y, y_type, M, N, ldy, st);
    if (int rc = check_matrix(W, S, "W")) return rc;
    if (int rc = check_rows(x, x_type, M, K, ldx, "x")) return rc;
    return product(W, S, 1, N, K, x_type, x, M, M > 1 ? ldx : K, nullptr, nullptr, M, y_type, y, M > 1 ? ldy : N, st);
}

int qmm_f8_experts(const void *W, const float *S, int64_t E, int64_t N, int64_t K, int x_type, const void *x, int64_t M,
                   int64_t ldx, const int32_t *offsets, const int32_t *rows, int64_t R, int y_type, void *y, int64_t ldy,
                   void *stream) {
    qk::clear_error();
    if (int rc = check_ftype(x_type, "x")) return rc;
    if (int rc = check_ftype(y_type, "y")) return rc;
    if (int rc = check_experts(E)) return rc;
    if (int rc = check_sizes(E, N, K, R)) return rc;
    if (M < 0 || M >= I31 || (!rows && M != R))
        return refuse(QMM_EINVAL_SHAPE, "M=%lld rows of x for R=%lld rows of y: equal without a row index",
                      static_cast<ll>(M), static_cast<ll>(R));
    if (R == 0 || N == 0) return QMM_OK;
    if (int rc = check_words(offsets, "offsets")) return rc;
    if (rows && !aligned(rows, 4)) return refuse(QMM_EINVAL_PTR, "rows must be 4-byte aligned");
    if (int rc = check_rows(y, y_type, R, N, ldy, "y")) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) return zero_rows(y, y_type, R, N, ldy, st);
    if (M == 0) return refuse(QMM_EINVAL_SHAPE, "R=%lld rows from an empty x", static_cast<ll>(R));
    if (int rc = check_matrix(W, S, "W")) return rc;
    if (int rc = check_rows(x, x_type, M, K, ldx, "x")) return rc;
    return product(W, S, E, N, K, x_type, x, M, M > 1 ? ldx : K, offsets, rows, R, y_type, y, R > 1 ? ldy : N, st);
}

int qmm_route(int x_type, const void *logits, int64_t T, int64_t E, int64_t ldx, int k, int score, int normalize,
              float factor, float *weights, int32_t *experts, int32_t *offsets, int32_t *rows, int32_t *slots,
              void *stream) {
    qk::clear_error();
    if (int rc = check_ftype(x_type, "logits")) return rc;
    if (int rc = check_experts(E)) return rc;
    if (k < 1 || k > QMM_ROUTE_MAX_K || k > E)
        return refuse(QMM_EINVAL_SHAPE, "k=%d: 1 to %d choices, at most E=%lld", k, QMM_ROUTE_MAX_K, static_cast<ll>(E));
    if (T < 0 || T >= I31 / k) return refuse(QMM_EINVAL_SHAPE, "T=%lld k=%d: 0 <= T*k < 2^31", static_cast<ll>(T), k);
    if (score != QMM_ROUTE_SOFTMAX && score != QMM_ROUTE_SIGMOID)
        return refuse(QMM_EINVAL_TYPE, "unknown score function %d", score);
    if (int rc = check_words(offsets, "offsets")) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        const cudaError_t e = cudaMemsetAsync(offsets, 0, static_cast<size_t>(E + 1) * 4, st);
        return e == cudaSuccess ? QMM_OK : cuda_error(e, "zero fill");
    }
    if (int rc = check_rows(logits, x_type, T, E, ldx, "logits")) return rc;
    if (int rc = check_words(weights, "weights")) return rc;
    if (int rc = check_words(experts, "experts")) return rc;
    if (int rc = check_words(rows, "rows")) return rc;
    if (int rc = check_words(slots, "slots")) return rc;
    qk::F8Context c;
    if (int rc = qk::f8_context(c)) return rc;
    const qk::CallLock lock(c.dev, st);
    void *hist = nullptr;
    if (const size_t bytes = qk::f8_route_hist_bytes(T, static_cast<int>(E), c.num_sms))
        if (int rc = qk::f8_workspace(c, st, bytes, &hist)) return rc;
    const qk::F8Route r = {x_type,  logits,  T,       T > 1 ? ldx : E, static_cast<int>(E), k,
                           score,   normalize, factor, weights, experts, offsets, rows, slots,
                           static_cast<int32_t *>(hist), c.dev};
    const cudaError_t e = qk::launch_f8_route(r, st, c.num_sms);
    if (e != cudaSuccess) return cuda_error(e, "route launch");
    qk::count_launches(qk::f8_route_launches(T, static_cast<int>(E), c.num_sms));
    return QMM_OK;
}

int qmm_f8_moe(int x_type, const void *x, int64_t T, int64_t H, int64_t ldx, int k, const float *weights,
               const int32_t *offsets, const int32_t *slots, int64_t E, int64_t I, const void *W_gate,
               const float *S_gate, const void *W_up, const float *S_up, const void *W_down, const float *S_down,
               int y_type, void *y, int64_t ldy, void *stream) {
    qk::clear_error();
    if (int rc = check_ftype(x_type, "x")) return rc;
    if (int rc = check_ftype(y_type, "y")) return rc;
    if (int rc = check_experts(E)) return rc;
    if (k < 1 || k > QMM_ROUTE_MAX_K || k > E)
        return refuse(QMM_EINVAL_SHAPE, "k=%d: 1 to %d choices, at most E=%lld", k, QMM_ROUTE_MAX_K, static_cast<ll>(E));
    if (T < 0 || T >= I31 / k) return refuse(QMM_EINVAL_SHAPE, "T=%lld k=%d: 0 <= T*k < 2^31", static_cast<ll>(T), k);
    const int64_t R = T * k;
    if (int rc = check_sizes(E, I, H, R)) return rc;
    if (int rc = check_sizes(E, H, I, R)) return rc;
    if (T == 0 || H == 0) return QMM_OK;
    if (int rc = check_rows(y, y_type, T, H, ldy, "y")) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (I == 0) return zero_rows(y, y_type, T, H, ldy, st);
    if (int rc = check_rows(x, x_type, T, H, ldx, "x")) return rc;
    if (int rc = check_words(weights, "weights")) return rc;
    if (int rc = check_words(offsets, "offsets")) return rc;
    if (int rc = check_words(slots, "slots")) return rc;
    if (int rc = check_matrix(W_gate, S_gate, "W_gate")) return rc;
    if (int rc = check_matrix(W_up, S_up, "W_up")) return rc;
    if (int rc = check_matrix(W_down, S_down, "W_down")) return rc;

    qk::F8Context c;
    if (int rc = qk::f8_context(c)) return rc;
    if (!qk::f8_available()) return refuse(QMM_ECUDA, "the driver has no tensor map encoder");
    const qk::CallLock lock(c.dev, st);
    // workspace: codes and scales of x per row | of h | the rows of
    // the down product in fp32 | partial tiles
    const Codes qx(R, H), qh(R, I);
    const int64_t ldd = up(H, 4);
    const size_t d_bytes = static_cast<size_t>(up(R * ldd * 4, 1024));
    const size_t part1 = qk::f8_part_bytes(R, static_cast<int>(E), I, true, true, c.num_sms);
    const size_t part2 = qk::f8_part_bytes(R, static_cast<int>(E), H, false, true, c.num_sms);
    const size_t part = part1 > part2 ? part1 : part2;
    char *at = nullptr;
    if (int rc = qk::f8_workspace(c, st, qx.q_bytes + qx.s_bytes + qh.q_bytes + qh.s_bytes + d_bytes + part,
                                  reinterpret_cast<void **>(&at)))
        return rc;
    unsigned *count = nullptr;
    if (int rc = qk::f8_counters(c, st, &count)) return rc;
    uint8_t *xq = reinterpret_cast<uint8_t *>(at);
    float *xs = reinterpret_cast<float *>(at += qx.q_bytes);
    uint8_t *hq = reinterpret_cast<uint8_t *>(at += qx.s_bytes);
    float *hs = reinterpret_cast<float *>(at += qh.q_bytes);
    float *d = reinterpret_cast<float *>(at += qh.s_bytes);
    float *partial = reinterpret_cast<float *>(at += d_bytes);

    qk::F8Quant f = {};
    f.x_type = x_type;
    f.x = x;
    f.M = T;
    f.K = H;
    f.ldx = T > 1 ? ldx : H;
    f.q = xq;
    f.ld_q = qx.ld;
    f.s = xs;
    f.s_row = 1;
    f.s_blk = qx.ld_s;
    f.map = slots;
    f.k = k;
    f.rows_max = R;
    f.status = c.status;
    f.dev = c.dev;
    cudaError_t e = qk::launch_f8_quantize(f, st, c.num_sms);
    if (e != cudaSuccess) return cuda_error(e, "quantize launch");
    qk::count_launches(1);

    qk::F8Gemm g = {};
    g.W = static_cast<const uint8_t *>(W_gate);
    g.W2 = static_cast<const uint8_t *>(W_up);
    g.Ws = S_gate;
    g.W2s = S_up;
    g.E = static_cast<int>(E);
    g.N = I;
    g.K = H;
    g.xq = xq;
    g.ld_q = qx.ld;
    g.xs = xs;
    g.ld_s = qx.ld_s;
    g.offsets = offsets;
    g.R = R;
    g.hq = hq;
    g.ld_h = qh.ld;
    g.hs = hs;
    g.ld_hs = qh.ld_s;
    g.part = partial;
    g.count = count;
    g.status = c.status;
    g.dev = c.dev;
    e = qk::launch_f8_gemm(g, st, c.num_sms);
    if (e != cudaSuccess) return cuda_error(e, "gate and up launch");
    qk::count_launches(1);

    g.W = static_cast<const uint8_t *>(W_down);
    g.W2 = nullptr;
    g.Ws = S_down;
    g.N = H;
    g.K = I;
    g.xq = hq;
    g.ld_q = qh.ld;
    g.xs = hs;
    g.ld_s = qh.ld_s;
    g.y_type = QMM_F32;
    g.y = d;
    g.ldy = ldd;
    e = qk::launch_f8_gemm(g, st, c.num_sms);
    if (e != cudaSuccess) return cuda_error(e, "down launch");
    qk::count_launches(1);

    e = qk::launch_f8_combine(d, ldd, R, weights, slots, T, k, H, y_type, y, T > 1 ? ldy : H, c.status, st, c.num_sms,
                              c.dev);
    if (e != cudaSuccess) return cuda_error(e, "weighted sum launch");
    qk::count_launches(1);
    return QMM_OK;
}

}  // extern "C"
