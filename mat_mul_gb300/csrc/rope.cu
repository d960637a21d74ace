// rope.cu -- position rotation: y = factor * R(position) x on the pairs of the
// first `rot` values of every head, the others copied.
//
// A pair (a, b) at angle w becomes (a cos w - b sin w, b cos w + a sin w), w =
// position * frequency of the pair; the transpose (the gradient) turns by -w.
// Bound by memory once there are a few hundred tokens, by latency below.  A
// thread owns a group of pairs of one token and takes it through several heads,
// so that the sines are paid once for them.  8191 x 40 x 128 bf16: 27.8 us, 0.89 of
// the rate of a copy.
#include "kv_device.cuh"

namespace qk {

namespace {

struct RopeParams {
    const void *x;
    void *y;
    int64_t T, ldx_t, ldx_h, ldy_t, ldy_h;
    int heads, groups, per;  // heads a thread takes
    const int32_t *positions;
    RopeArgs rope;
};

constexpr int ROPE_THREADS = 128;

template <int TX, int TY, int V>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const RopeParams P) {
    using X = typename KvElem<TX>::type;
    using Y = typename KvElem<TY>::type;
    constexpr int BATCH = 4;
    pdl_wait();
    pdl_trigger();
    const int parts = (P.heads + P.per - 1) / P.per;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * ROPE_THREADS + threadIdx.x;
    const int64_t tp = n / P.groups;
    const int g = static_cast<int>(n - tp * P.groups);
    const int64_t t = tp / parts;
    if (t >= P.T) return;
    const int h0 = static_cast<int>(tp - t * parts) * P.per, h1 = min(P.heads, h0 + P.per);
    const Group<V> group(g, P.rope);
    float2 cs[V];
    group.angles(P.rope, __ldg(P.positions + t), cs);
    const X *x = static_cast<const X *>(P.x) + t * P.ldx_t + h0 * P.ldx_h;
    Y *y = static_cast<Y *>(P.y) + t * P.ldy_t + h0 * P.ldy_h;
    turn_heads<X, Y, V, BATCH>(x, P.ldx_h, y, P.ldy_h, h1 - h0, group, cs);
}

bool runs_of(const Heads &a, int64_t T, int heads, int v) {
    const int64_t bytes = v * f8_size(a.type);
    auto whole = [&](int64_t ld) { return ld * f8_size(a.type) % bytes == 0; };
    return reinterpret_cast<uintptr_t>(a.x) % bytes == 0 && (T == 1 || whole(a.ld_t)) && (heads == 1 || whole(a.ld_h));
}

template <int TX, int TY, int V>
cudaError_t launch_one(const KvRope &r, cudaStream_t st, int num_sms) {
    RopeParams p = {};
    p.x = r.x.x;
    p.y = const_cast<void *>(r.y.x);
    p.T = r.T;
    p.ldx_t = r.x.ld_t, p.ldx_h = r.x.ld_h, p.ldy_t = r.y.ld_t, p.ldy_h = r.y.ld_h;
    p.heads = r.heads;
    p.groups = (r.dim + 2 * V - 1) / (2 * V);
    p.positions = r.positions;
    p.rope = r.rope;
    // as many heads per thread as leave every multiprocessor 2048 threads
    const int64_t all = r.T * r.heads * p.groups, want = static_cast<int64_t>(num_sms) * 2048;
    p.per = static_cast<int>(all / want < 1 ? 1 : all / want > 8 ? 8 : all / want);
    const int64_t parts = (r.heads + p.per - 1) / p.per;
    const int64_t blocks = (r.T * parts * p.groups + ROPE_THREADS - 1) / ROPE_THREADS;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(ROPE_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_kernel<TX, TY, V>, p);
}

template <int TX, int TY>
cudaError_t launch_v(const KvRope &r, cudaStream_t st, int num_sms) {
    constexpr int W = TX == QMM_F32 || TY == QMM_F32 ? 4 : 8;
    auto fits = [&](int v) {
        return r.rope.rot % (2 * v) == 0 && r.dim % (2 * v) == 0 && runs_of(r.x, r.T, r.heads, v) && runs_of(r.y, r.T, r.heads, v);
    };
    if (fits(W)) return launch_one<TX, TY, W>(r, st, num_sms);
    if (W > 4 && fits(4)) return launch_one<TX, TY, 4>(r, st, num_sms);
    return launch_one<TX, TY, 1>(r, st, num_sms);
}

template <int TX>
cudaError_t launch_y(const KvRope &r, cudaStream_t st, int num_sms) {
    if (r.y.type == QMM_F32) return launch_v<TX, QMM_F32>(r, st, num_sms);
    if (r.y.type == QMM_F16) return launch_v<TX, QMM_F16>(r, st, num_sms);
    return launch_v<TX, QMM_BF16>(r, st, num_sms);
}

}  // namespace

cudaError_t launch_rope(const KvRope &r, cudaStream_t st, int num_sms) {
    if (r.x.type == QMM_F32) return launch_y<QMM_F32>(r, st, num_sms);
    if (r.x.type == QMM_F16) return launch_y<QMM_F16>(r, st, num_sms);
    return launch_y<QMM_BF16>(r, st, num_sms);
}

}  // namespace qk
