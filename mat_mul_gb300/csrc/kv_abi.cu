// kv_abi.cu -- C entry points of the position rotation and of the paged key and
// value cache: argument checks, scratch and launches.
#include <cmath>

#include "abi_checks.h"
#include "kv_internal.h"

namespace {

int check_values(const void *p, int type, const char *what) {
    if (!p) return refuse(QMM_EINVAL_PTR, "%s is null", what);
    if (!aligned(p, qk::f8_size(type)))
        return refuse(QMM_EINVAL_PTR, "%s must be aligned to its values (%d bytes)", what, qk::f8_size(type));
    return QMM_OK;
}

int check_type64(int64_t t, const char *what) {
    return t < 0 || t > QMM_BF16 ? refuse(QMM_EINVAL_TYPE, "%s: unknown value type %lld", what, static_cast<ll>(t))
                                 : check_ftype(static_cast<int>(t), what);
}

// Rows of heads that are written: no element may belong to two of them.
int check_apart(int64_t T, int64_t heads, int64_t dim, int64_t ld_t, int64_t ld_h, const char *what) {
    int64_t n[2] = {T, heads}, ld[2] = {ld_t, ld_h}, extent = dim;
    const int first = heads <= 1 || (T > 1 && ld_t < ld_h) ? 0 : 1;  // the smaller pitch first
    for (int i = 0; i < 2; ++i) {
        const int k = i ? 1 - first : first;
        if (n[k] <= 1) continue;
        if (ld[k] < extent)
            return refuse(QMM_EINVAL_SHAPE, "%s: heads or rows overlap (pitches %lld and %lld)", what, static_cast<ll>(ld_t),
                          static_cast<ll>(ld_h));
        extent += (n[k] - 1) * ld[k];
    }
    return QMM_OK;
}

int check_rope(const qmm_rope_table *r, int64_t dim, qk::RopeArgs &out) {
    if (r->rot < 0 || r->rot % 2 || r->rot > dim)
        return refuse(QMM_EINVAL_SHAPE, "rotation of %lld values of a head of %lld: even and no more than the head",
                      static_cast<ll>(r->rot), static_cast<ll>(dim));
    if (r->rot && !r->turns) return refuse(QMM_EINVAL_PTR, "turns is null");
    if (!aligned(r->turns, 8)) return refuse(QMM_EINVAL_PTR, "turns must be 8-byte aligned");
    out.turns = r->turns;
    out.rot = static_cast<int>(r->rot);
    out.interleaved = r->interleaved != 0;
    out.inverse = 0;
    out.factor = static_cast<float>(r->factor);
    return QMM_OK;
}

int check_cache(const qmm_kv_cache *c) {
    if (!c) return refuse(QMM_EINVAL_PTR, "cache is null");
    if (c->heads < 1 || c->heads > 1024 || c->pages < 0 || c->pages >= I31)
        return refuse(QMM_EINVAL_SHAPE, "cache of %lld pages and %lld heads: 1 to 1024 heads, fewer than 2^31 pages",
                      static_cast<ll>(c->pages), static_cast<ll>(c->heads));
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
        return refuse(QMM_EINVAL_SHAPE, "pages of %lld tokens: 16, 32, 64 or 128", static_cast<ll>(c->page));
    if (c->dim < 16 || c->dim > 256 || c->dim % 16)
        return refuse(QMM_EINVAL_SHAPE, "heads of %lld values: a multiple of 16 up to 256", static_cast<ll>(c->dim));
    return QMM_OK;
}
// What a call with rows needs besides.
int check_pages(const qmm_kv_cache *c) {
    if (c->pages < 1) return refuse(QMM_EINVAL_SHAPE, "a cache without pages");
    if (c->pages * c->heads >= I31)    // (page, head) is one coordinate of a tensor map
        return refuse(QMM_EINVAL_SHAPE, "cache of %lld pages and %lld heads: pages * heads must be below 2^31",
                      static_cast<ll>(c->pages), static_cast<ll>(c->heads));
    if (!c->k || !c->v) return refuse(QMM_EINVAL_PTR, "cache: codes are null");
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return refuse(QMM_EINVAL_PTR, "cache: codes must be 16-byte aligned");
    if (int rc = check_words(c->k_scale, "cache: key scales")) return rc;
    return check_words(c->v_scale, "cache: value scales");
}

template <class Args>
int check_batch(const Args &a, qk::KvBatch &out) {
    if (a.T < 0 || a.T >= I31 || a.B < 0 || a.B >= I31 / 4 || a.width < 0)
        return refuse(QMM_EINVAL_SHAPE, "T=%lld B=%lld width=%lld: out of range", static_cast<ll>(a.T), static_cast<ll>(a.B),
                      static_cast<ll>(a.width));
    if (!a.offsets && a.T != a.B)
        return refuse(QMM_EINVAL_SHAPE, "T=%lld rows of B=%lld sequences: equal without offsets", static_cast<ll>(a.T),
                      static_cast<ll>(a.B));
    if (a.width > (I31 - 256) / a.cache->page)
        return refuse(QMM_EINVAL_SHAPE, "width=%lld pages of %lld tokens: below 2^31 tokens a sequence",
                      static_cast<ll>(a.width), static_cast<ll>(a.cache->page));
    if (a.B > 1 && a.ld_table < a.width)
        return refuse(QMM_EINVAL_SHAPE, "table: a row pitch of %lld is less than its %lld entries", static_cast<ll>(a.ld_table),
                      static_cast<ll>(a.width));
    if (a.B == 0 || a.T == 0) return QMM_OK;
    if (int rc = check_words(a.lengths, "lengths")) return rc;
    if (!aligned(a.offsets, 4)) return refuse(QMM_EINVAL_PTR, "offsets must be 4-byte aligned");
    if (a.width > 0)
        if (int rc = check_words(a.table, "table")) return rc;
    out.offsets = a.offsets;
    out.lengths = a.lengths;
    out.table = a.table;
    out.ld_table = a.B > 1 ? a.ld_table : a.width;
    out.width = static_cast<int>(a.width);
    out.B = static_cast<int>(a.B);
    out.T = a.T;
    return QMM_OK;
}

int check_attention(const qmm_kv_attention_args *args, qk::KvAttention &out) {
    if (!args) return refuse(QMM_EINVAL_PTR, "args is null");
    const qmm_kv_attention_args &a = *args;
    if (int rc = check_cache(a.cache)) return rc;
    if (int rc = check_type64(a.q_type, "q")) return rc;
    if (int rc = check_type64(a.y_type, "y")) return rc;
    if (a.q_heads < 1 || a.q_heads > 16384 || a.q_heads % a.cache->heads)
        return refuse(QMM_EINVAL_SHAPE, "q_heads=%lld: a multiple of the cache's %lld heads, up to 16384",
                      static_cast<ll>(a.q_heads), static_cast<ll>(a.cache->heads));
    if (a.window < 0 || (a.window && !a.causal))
        return refuse(QMM_EINVAL_SHAPE, "window=%lld: at least 0, and 0 unless causal", static_cast<ll>(a.window));
    if (!std::isfinite(a.scale) || std::fabs(a.scale) > 1e30)
        return refuse(QMM_EINVAL_SHAPE, "scale=%g: finite, at most 1e30", a.scale);
    if (int rc = check_batch(a, out.batch)) return rc;
    if (a.T * (a.q_heads / a.cache->heads) >= I31 - 256)
        return refuse(QMM_EINVAL_SHAPE, "T=%lld rows of %lld heads: too large", static_cast<ll>(a.T), static_cast<ll>(a.q_heads));
    out.c = *a.cache;
    out.q = {a.q, a.ldq_t, a.ldq_h, static_cast<int>(a.q_type)};
    out.y = {a.y, a.ldy_t, a.ldy_h, static_cast<int>(a.y_type)};
    out.q_heads = static_cast<int>(a.q_heads);
    out.scale = a.scale;
    out.causal = a.causal != 0;
    out.window = a.window >= I31 ? 0 : static_cast<int>(a.window);  // (no sequence is longer)
    out.lse = a.lse;
    return QMM_OK;
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

extern "C" {

int qmm_rope_turns(int rot, double base, const double *freqs, int scaling, double scale, double original, double low,
                   double high, uint64_t *turns) {
    qk::clear_error();
    constexpr double TWO_PI = 6.283185307179586476925286766559;
    if (rot < 0 || rot % 2) return refuse(QMM_EINVAL_SHAPE, "rot=%d: even and at least 0", rot);
    if (scaling < QMM_ROPE_PLAIN || scaling > QMM_ROPE_PARTS) return refuse(QMM_EINVAL_TYPE, "unknown scaling %d", scaling);
    if (!freqs && !(base > 0 && std::isfinite(base))) return refuse(QMM_EINVAL_SHAPE, "base=%g: positive", base);
    if (scaling != QMM_ROPE_PLAIN && !(scale > 0 && std::isfinite(scale)))
        return refuse(QMM_EINVAL_SHAPE, "scale=%g: positive", scale);
    if (scaling == QMM_ROPE_NTK && (freqs || rot < 4))
        return refuse(QMM_EINVAL_SHAPE, "the NTK scaling changes the base: no frequencies of your own, rot=%d at least 4", rot);
    if (scaling == QMM_ROPE_PARTS && !(original > 0 && std::isfinite(original) && high > low && std::isfinite(high - low)))
        return refuse(QMM_EINVAL_SHAPE, "original=%g low=%g high=%g: original positive, low < high", original, low, high);
    if (rot && !turns) return refuse(QMM_EINVAL_PTR, "turns is null");
    if (scaling == QMM_ROPE_NTK) base *= std::pow(scale, rot / (rot - 2.0));
    for (int i = 0; i < rot / 2; ++i) {
        double f = freqs ? freqs[i] : std::pow(base, -2.0 * i / rot);
        if (scaling == QMM_ROPE_LINEAR) f /= scale;
        if (scaling == QMM_ROPE_PARTS) {
            double k = (original * f / TWO_PI - low) / (high - low);
            k = k < 0 ? 0 : k > 1 ? 1 : k;
            f = f * k + f / scale * (1 - k);
        }
        if (!std::isfinite(f)) return refuse(QMM_EINVAL_SHAPE, "frequency %d is %g", i, f);
        double part = f / TWO_PI;  // whole turns do not matter, positions are whole numbers
        part -= std::floor(part);
        const double v = std::nearbyint(std::ldexp(part, 64));
        turns[i] = v >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(v);
    }
    return QMM_OK;
}

int qmm_rope(const qmm_rope_args *args, void *stream) {
    qk::clear_error();
    if (!args) return refuse(QMM_EINVAL_PTR, "args is null");
    const qmm_rope_args &a = *args;
    if (int rc = check_type64(a.x_type, "x")) return rc;
    if (int rc = check_type64(a.y_type, "y")) return rc;
    if (a.T < 0 || a.T >= I31 || a.heads < 0 || a.heads > 65536 || a.dim < 0 || a.dim > 65536 || a.dim % 2)
        return refuse(QMM_EINVAL_SHAPE, "T=%lld heads=%lld dim=%lld: T below 2^31, up to 65536 heads, dim even up to 65536",
                      static_cast<ll>(a.T), static_cast<ll>(a.heads), static_cast<ll>(a.dim));
    if (!a.rope) return refuse(QMM_EINVAL_PTR, "rope is null");
    qk::KvRope r = {};
    if (int rc = check_rope(a.rope, a.dim, r.rope)) return rc;
    if (a.T == 0 || a.heads == 0 || a.dim == 0) return QMM_OK;
    if (a.T * a.heads >= I31) return refuse(QMM_EINVAL_SHAPE, "T=%lld heads=%lld: too large", static_cast<ll>(a.T), static_cast<ll>(a.heads));
    if (int rc = check_words(a.positions, "positions")) return rc;
    if (int rc = check_values(a.x, static_cast<int>(a.x_type), "x")) return rc;
    if (int rc = check_values(a.y, static_cast<int>(a.y_type), "y")) return rc;
    if (int rc = check_apart(a.T, a.heads, a.dim, a.ldy_t, a.ldy_h, "y")) return rc;
    if (a.x == a.y && (a.x_type != a.y_type || (a.T > 1 && a.ldx_t != a.ldy_t) || (a.heads > 1 && a.ldx_h != a.ldy_h)))
        return refuse(QMM_EINVAL_SHAPE, "y is x: it needs the same type and pitches");
    qk::F8Context c;
    if (int rc = qk::f8_context(c)) return rc;
    r.rope.inverse = a.inverse != 0;
    r.x = {a.x, a.ldx_t, a.ldx_h, static_cast<int>(a.x_type)};
    r.y = {a.y, a.ldy_t, a.ldy_h, static_cast<int>(a.y_type)};
    r.T = a.T;
    r.heads = static_cast<int>(a.heads);
    r.dim = static_cast<int>(a.dim);
    r.positions = a.positions;
    const cudaError_t e = qk::launch_rope(r, static_cast<cudaStream_t>(stream), c.num_sms);
    if (e != cudaSuccess) return cuda_error(e, "rotation launch");
    qk::count_launches(1);
    return QMM_OK;
}

int qmm_kv_append(const qmm_kv_append_args *args, void *stream) {
    qk::clear_error();
    if (!args) return refuse(QMM_EINVAL_PTR, "args is null");
    const qmm_kv_append_args &a = *args;
    if (int rc = check_cache(a.cache)) return rc;
    if (int rc = check_type64(a.x_type, "k")) return rc;
    const int type = static_cast<int>(a.x_type);
    qk::KvAppend r = {};
    if (int rc = check_batch(a, r.batch)) return rc;
    if (a.rope)
        if (int rc = check_rope(a.rope, a.cache->dim, r.rope)) return rc;
    if (a.q) {
        if (a.q_heads < 1 || a.q_heads > 16384)
            return refuse(QMM_EINVAL_SHAPE, "q_heads=%lld: 1 to 16384", static_cast<ll>(a.q_heads));
        if (!a.rope) return refuse(QMM_EINVAL_PTR, "queries without a rotation");
    }
    if (a.B == 0 || a.T == 0) return QMM_OK;
    if (int rc = check_pages(a.cache)) return rc;
    if (int rc = check_values(a.k, type, "k")) return rc;
    if (int rc = check_values(a.v, type, "v")) return rc;
    if (!aligned(a.positions, 4)) return refuse(QMM_EINVAL_PTR, "positions must be 4-byte aligned");
    if (a.q) {
        if (int rc = check_values(a.q, type, "q")) return rc;
        if (int rc = check_values(a.q_out, type, "q_out")) return rc;
        if (int rc = check_apart(a.T, a.q_heads, a.cache->dim, a.ldo_t, a.ldo_h, "q_out")) return rc;
        if (a.q == a.q_out && ((a.T > 1 && a.ldq_t != a.ldo_t) || (a.q_heads > 1 && a.ldq_h != a.ldo_h)))
            return refuse(QMM_EINVAL_SHAPE, "q_out is q: it needs the same pitches");
    }
    qk::F8Context c;
    if (int rc = qk::f8_context(c)) return rc;
    r.c = *a.cache;
    r.k = {a.k, a.ldk_t, a.ldk_h, type};
    r.v = {a.v, a.ldv_t, a.ldv_h, type};
    r.q = {a.q, a.ldq_t, a.ldq_h, type};
    r.y = {a.q_out, a.ldo_t, a.ldo_h, type};
    r.q_heads = static_cast<int>(a.q_heads);
    r.positions = a.positions;
    r.status = c.status;
    const cudaError_t e = qk::launch_kv_append(r, static_cast<cudaStream_t>(stream), c.num_sms);
    if (e != cudaSuccess) return cuda_error(e, "append launch");
    qk::count_launches(1);
    return QMM_OK;
}

int64_t qmm_kv_attention_scratch(const qmm_kv_attention_args *args) {
    qk::clear_error();
    qk::KvAttention r = {};
    if (int rc = check_attention(args, r)) return rc;
    if (args->B == 0 || args->T == 0) return 0;
    qk::F8Context c;
    if (int rc = qk::f8_context(c)) return rc;
    const qk::KvPlan plan = qk::kv_attention_plan(r, c.num_sms);
    return static_cast<int64_t>(up256(plan.scratch) + up256(static_cast<size_t>(plan.counters) * 4));
}

int qmm_kv_attention(const qmm_kv_attention_args *args, void *stream) {
    qk::clear_error();
    qk::KvAttention r = {};
    if (int rc = check_attention(args, r)) return rc;
    const qmm_kv_attention_args &a = *args;
    if (a.B == 0 || a.T == 0) return QMM_OK;
    if (int rc = check_pages(a.cache)) return rc;
    if (int rc = check_values(a.q, r.q.type, "q")) return rc;
    if (int rc = check_values(a.y, r.y.type, "y")) return rc;
    if (int rc = check_apart(a.T, a.q_heads, a.cache->dim, a.ldy_t, a.ldy_h, "y")) return rc;
    if (a.q == a.y) return refuse(QMM_EINVAL_PTR, "y is q: blocks that share a row's tokens read q while others write y");
    if (a.lse && !aligned(a.lse, 4)) return refuse(QMM_EINVAL_PTR, "lse must be 4-byte aligned");
    qk::F8Context c;
    if (int rc = qk::f8_context(c)) return rc;
    if (!qk::f8_available()) return refuse(QMM_ECUDA, "the driver has no tensor map encoder");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const qk::CallLock lock(c.dev, st);
    const qk::KvPlan plan = qk::kv_attention_plan(r, c.num_sms);
    if (a.scratch) {
        const size_t part = up256(plan.scratch), words = static_cast<size_t>(plan.counters) * 4;
        if (!aligned(a.scratch, 256)) return refuse(QMM_EINVAL_PTR, "scratch must be 256-byte aligned");
        if (a.scratch_bytes < 0 || static_cast<size_t>(a.scratch_bytes) < part + words)
            return refuse(QMM_EINVAL_SHAPE, "scratch of %lld bytes, %zu needed", static_cast<ll>(a.scratch_bytes), part + words);
        r.scratch = static_cast<char *>(a.scratch);
        r.count = reinterpret_cast<unsigned *>(r.scratch + part);
        if (words) {
            const cudaError_t e = cudaMemsetAsync(r.count, 0, words, st);
            if (e != cudaSuccess) return cuda_error(e, "counters init");
        }
    } else {
        if (plan.scratch)
            if (int rc = qk::f8_workspace(c, st, plan.scratch, reinterpret_cast<void **>(&r.scratch))) return rc;
        if (plan.counters)
            if (int rc = qk::f8_counters_n(c, st, plan.counters, &r.count)) return rc;
    }
    r.status = c.status;
    r.dev = c.dev;
    r.stop = qk::inject_stop_stage();
    const cudaError_t e = qk::launch_kv_attention(r, st, c.num_sms);
    if (e != cudaSuccess) return cuda_error(e, "attention launch");
    qk::count_launches(1);
    return QMM_OK;
}

}  // extern "C"
