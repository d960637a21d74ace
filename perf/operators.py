"""Measured cases of the block-scaled 8-bit-float products and the expert layer built on them.

Every operator in two forms: the framework's (own = True) and a plain one from elementary
torch operations in 32 bits.  Sizes follow the shapes the repository benchmarks (Llama-3.2-1B,
Mistral-7B, Qwen3-14B projections); the expert shapes are generic.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
B = 128          # weights and activations carry one scale per 128 (x 128) values
TOP = 448.0      # the largest e4m3 value
TINY = 2.0 ** -126


def listed():
    return [
        # one decode step's activations, a few concurrent requests, before a Mistral-7B projection
        {"name": "quantize 4x4096 bf16", "op": "quantize", "M": 4, "K": 4096, "x": "bf16", "pad": 0},
        # a long prefill's activations at Qwen3-14B's hidden size, an odd number of tokens
        {"name": "quantize 8191x5120 bf16", "op": "quantize", "M": 8191, "K": 5120, "x": "bf16", "pad": 0},
        # one token through Mistral-7B's up projection: weight streaming
        {"name": "f8 1x4096x14336 bf16", "op": "f8", "M": 1, "K": 4096, "N": 14336, "x": "bf16", "y": "bf16", "pad": 0},
        # a small batch through Qwen3-14B's k projection: little work, latency counts
        {"name": "f8 13x5120x1024 f16", "op": "f8", "M": 13, "K": 5120, "N": 1024, "x": "f16", "y": "f16", "pad": 0},
        # a ragged prefill chunk: no size a multiple of 128, rows of x further apart than K, float32 in and out
        {"name": "f8 509x2064x5000 f32", "op": "f8", "M": 509, "K": 2064, "N": 5000, "x": "f32", "y": "f32", "pad": 12},
        # a full prefill batch through Qwen3-14B's gate projection: tensor-core bound
        {"name": "f8 4096x5120x17408 bf16", "op": "f8", "M": 4096, "K": 5120, "N": 17408, "x": "bf16", "y": "bf16",
         "pad": 0},
        # sixteen decoding tokens, four experts each: most experts see one row or none
        {"name": "experts 64 rows E64 bf16", "op": "experts", "T": 16, "k": 4, "E": 64, "A": 41, "K": 2048, "N": 1536,
         "x": "bf16", "y": "bf16", "gather": True},
        # a prefill's rows over experts of very different load, some without any
        {"name": "experts 8192 rows E40 bf16", "op": "experts", "T": 2048, "k": 4, "E": 40, "A": 37, "K": 2048,
         "N": 2880, "x": "bf16", "y": "bf16", "gather": False},
        # the router of one decode step
        {"name": "route 8 tokens E128 f32", "op": "route", "T": 8, "E": 128, "k": 8, "x": "f32", "score": "softmax",
         "norm": True, "masked": 0},
        # the router of a long prefill, sigmoid scores, two experts masked out
        {"name": "route 16384 tokens E64 bf16", "op": "route", "T": 16384, "E": 64, "k": 6, "x": "bf16",
         "score": "sigmoid", "norm": True, "masked": 2},
        # an expert layer in decode: four tokens, the weights of the chosen experts are what is read
        {"name": "moe 4 tokens E64 bf16", "op": "moe", "T": 4, "k": 6, "E": 64, "A": 21, "H": 2048, "I": 1024,
         "x": "bf16", "y": "bf16"},
        # an expert layer in prefill, an odd number of tokens, experts of different load
        {"name": "moe 4093 tokens E32 bf16", "op": "moe", "T": 4093, "k": 4, "E": 32, "A": 32, "H": 2048, "I": 1408,
         "x": "bf16", "y": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "f8", "f8", "f8", "experts", "experts", "route", "moe", "moe"])
    x = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        return {"op": op, "M": _log(rng, 1, 8191), "K": _log(rng, 64, 5120), "x": x, "pad": rng.choice([0, 0, 8, 5])}
    if op == "f8":
        M = _log(rng, 1, 4096)
        return {"op": op, "M": M, "K": 16 * _log(rng, 8, 320 if M > 512 else 1088), "N": _log(rng, 64, 17408), "x": x,
                "y": rng.choice([x, x, "bf16", "f32"]), "pad": rng.choice([0, 0, 8, 5])}
    if op == "route":
        E = _log(rng, 4, 512)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E // 2, 10)), "x": x,
                "score": rng.choice(["softmax", "sigmoid"]), "norm": rng.random() < 0.7,
                "masked": rng.choice([0, 0, E // 4])}
    E = _log(rng, 4, 96)
    T = _log(rng, 1, 2048)
    k = rng.randint(1, min(E // 2, 8))
    A = min(T * k, rng.randint(max(k, E // 2), E))
    if op == "experts":
        return {"op": op, "T": T, "k": k, "E": E, "A": A, "K": 16 * _log(rng, 16, 128), "N": _log(rng, 96, 2880),
                "x": x, "y": rng.choice([x, "bf16", "f32"]), "gather": rng.random() < 0.5}
    # the intermediate activations are rounded to 8 bits between the products, so a float32 result is no sharper
    # than a 16-bit one
    x = rng.choice(["bf16", "f16"])
    return {"op": op, "T": T, "k": k, "E": E, "A": A, "H": 16 * _log(rng, 16, 128), "I": 16 * _log(rng, 8, 88), "x": x,
            "y": x}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _activations(g, M, K, kind, pad=0):
    """Unit normal activations, one value in a hundred twenty times larger; rows K + pad apart."""
    x = torch.randn(M, K + pad, generator=g, device="cuda")
    x *= 1.0 + 19.0 * (torch.rand(M, K + pad, generator=g, device="cuda") < 0.01)
    return x.to(TYPES[kind])[:, :K]


def _weights(g, E, N, K):
    """[E, N, K] codes and [E, ceil(N/128), ceil(K/128)] scales, as a checkpoint holds them."""
    nb, kb = -(-N // B), -(-K // B)
    W = torch.empty(E, N, K, dtype=FP8, device="cuda")
    S = torch.empty(E, nb, kb, device="cuda")
    for e in range(E):
        w = torch.zeros(nb * B, kb * B, device="cuda")
        w[:N, :K] = torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)
        t = w.view(nb, B, kb, B)
        S[e] = t.abs().amax(dim=(1, 3)) / TOP
        W[e] = (t / S[e][:, None, :, None]).view(nb * B, kb * B)[:N, :K].to(FP8)
    return W, S


def _pairs(g, c):
    """experts [T, k] with rows for exactly the A experts in use (small batches) or a skewed load over them."""
    T, k, E, A = c["T"], c["k"], c["E"], c["A"]
    use = torch.randperm(E, generator=g, device="cuda")[:A]
    if T * k <= 4 * A:
        flat = torch.arange(T * k, device="cuda") % A
        return use[flat].view(T, k)
    score = torch.randn(T, A, generator=g, device="cuda") + torch.randn(1, A, generator=g, device="cuda")
    return use[torch.topk(score, k, dim=1).indices]


def _sorted_pairs(experts, E):
    """The pairs (t, j) in expert order: offsets [E+1], token of each row, row of each pair, and the largest group."""
    flat = experts.reshape(-1)
    k = experts.shape[1]
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(order.numel(), device="cuda")
    return offsets, (order // k).to(torch.int32), slots.to(torch.int32).view_as(experts), int(counts.max())


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "quantize":
        s["x"] = _activations(g, c["M"], c["K"], c["x"], c["pad"])
    elif c["op"] == "f8":
        s["x"] = _activations(g, c["M"], c["K"], c["x"], c["pad"])
        W, S = _weights(g, 1, c["N"], c["K"])
        s["W"], s["S"] = W[0], S[0]
    elif c["op"] == "route":
        x = torch.randn(c["T"], c["E"], generator=g, device="cuda") * 2 + torch.randn(c["E"], generator=g, device="cuda")
        if c["masked"]:
            x[:, torch.randperm(c["E"], generator=g, device="cuda")[:c["masked"]]] = -math.inf
        s["x"] = x.to(TYPES[c["x"]])
    else:
        experts = _pairs(g, c)
        s["offsets"], s["rows"], s["slots"], s["most"] = _sorted_pairs(experts, c["E"])
        s["experts"] = experts.to(torch.int32)
        if c["op"] == "experts":
            s["x"] = _activations(g, c["T"] if c["gather"] else c["T"] * c["k"], c["K"], c["x"])
            s["W"], s["S"] = _weights(g, c["E"], c["N"], c["K"])
        else:
            s["x"] = _activations(g, c["T"], c["H"], c["x"])
            w = torch.rand(c["T"], c["k"], generator=g, device="cuda") + 0.1
            s["weights"] = w / w.sum(dim=1, keepdim=True)
            s["Wg"], s["Sg"] = _weights(g, c["E"], c["I"], c["H"])
            s["Wu"], s["Su"] = _weights(g, c["E"], c["I"], c["H"])
            s["Wd"], s["Sd"] = _weights(g, c["E"], c["H"], c["I"])
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _quantize(x):
    M, K = x.shape
    kb = -(-K // B)
    t = torch.zeros(M, kb * B, device=x.device)
    t[:, :K] = x
    t = t.view(M, kb, B)
    top = torch.full((), TOP, device=x.device)  # a division by a number would multiply by its rounded reciprocal
    s = (t.abs().amax(dim=2) / top).clamp(min=TINY)
    q = (t * (1.0 / s)[:, :, None]).to(FP8).view(M, kb * B)[:, :K]
    return q, s


def _rounded(x):
    """x [M, K] as the values its 8-bit codes stand for."""
    q, s = _quantize(x)
    return q.float() * s.repeat_interleave(B, dim=1)[:, :x.shape[1]]


def _dequantized(W, S):
    """[..., N, K] codes times their block's scale, in 32 bits."""
    s = S.repeat_interleave(B, dim=-2)[..., :W.shape[-2], :].repeat_interleave(B, dim=-1)[..., :W.shape[-1]]
    return W.float() * s


def _grouped(W, S, x, offsets, most):
    """y[r] = W[e] x[r] for the rows r of each expert e: one batched product over groups padded to `most` rows."""
    R = x.shape[0]
    lane = torch.arange(most, device=x.device)
    at = (offsets[:-1, None] + lane[None, :]).long()
    y = torch.bmm(x[at.clamp(max=R - 1)], _dequantized(W, S).transpose(1, 2))
    r = torch.arange(R, device=x.device)
    e = (r[:, None] >= offsets[None, 1:]).sum(dim=1)
    return y[e, r - offsets[e]]


def _route(x, k, score, norm):
    x = x.float()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    T, E = x.shape
    v, i = torch.sort(x, dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    if score == "softmax":
        m = v[:, :1]
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        w = torch.exp(v - m)
        total = w.sum(dim=1, keepdim=True) if norm else torch.exp(x - m).sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    else:
        w = 1.0 / (1.0 + torch.exp(-v))
        if norm:
            total = w.sum(dim=1, keepdim=True)
            w = torch.where(total > 0, w / total, torch.zeros_like(w))
    flat = i.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = (flat[:, None] == torch.arange(E, device=x.device)[None, :]).sum(dim=0)
    offsets = torch.cat([torch.zeros_like(counts[:1]), torch.cumsum(counts, 0)])
    slots = torch.empty_like(order)
    slots[order] = torch.arange(order.numel(), device=x.device)
    i32 = torch.int32
    return w, i.to(i32), offsets.to(i32), (order // k).to(i32), slots.view(T, k).to(i32)


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import mat_mul_gb300 as q
        if op == "quantize":
            return q.qmm_f8_quantize(s["x"])
        if op == "f8":
            return q.qmm_f8(s["W"], s["S"], s["x"], dtype=TYPES[c["y"]])
        if op == "route":
            r = q.qmm_route(s["x"], c["k"], score=c["score"], normalize=c["norm"])
            return r.weights, r.experts, r.offsets, r.rows, r.slots
        if op == "experts":
            return q.qmm_f8_experts(s["W"], s["S"], s["x"], s["offsets"], rows=s["rows"] if c["gather"] else None,
                                    dtype=TYPES[c["y"]])
        r = q.Route(s["weights"], s["experts"], s["offsets"], s["rows"], s["slots"])
        return q.qmm_f8_moe(s["x"], r, s["Wg"], s["Sg"], s["Wu"], s["Su"], s["Wd"], s["Sd"])
    if op == "quantize":
        return _quantize(s["x"])
    if op == "f8":
        return (_rounded(s["x"]) @ _dequantized(s["W"], s["S"]).t()).to(TYPES[c["y"]])
    if op == "route":
        return _route(s["x"], c["k"], c["score"], c["norm"])
    x = _rounded(s["x"])
    if op == "experts":
        if c["gather"]:
            x = x[s["rows"].long()]
        return _grouped(s["W"], s["S"], x, s["offsets"], s["most"]).to(TYPES[c["y"]])
    x = x[s["rows"].long()]
    gate = _grouped(s["Wg"], s["Sg"], x, s["offsets"], s["most"])
    up = _grouped(s["Wu"], s["Su"], x, s["offsets"], s["most"])
    h = _rounded(gate / (1.0 + torch.exp(-gate)) * up)
    y = _grouped(s["Wd"], s["Sd"], h, s["offsets"], s["most"])
    return (y[s["slots"].long()] * s["weights"][:, :, None]).sum(dim=1).to(TYPES[c["y"]])


# ---------------------------------------------------------------------------
# The least work, and the definition in 64 bits
# ---------------------------------------------------------------------------
def _weight_bytes(N, K):
    return N * K + 4 * (-(-N // B)) * (-(-K // B))


def work(case):
    c = case
    if c["op"] == "quantize":
        return {"bytes": c["M"] * c["K"] * (SIZE[c["x"]] + 1) + 4 * c["M"] * -(-c["K"] // B), "flops": 2 * c["M"] * c["K"]}
    if c["op"] == "f8":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": _weight_bytes(N, K) + M * (K * SIZE[c["x"]] + N * SIZE[c["y"]]), "flops": 2 * M * N * K}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * SIZE[c["x"]] + 16 * T * k + 4 * (E + 1), "flops": 4 * T * E}
    T, k, A = c["T"], c["k"], c["A"]
    R = T * k
    if c["op"] == "experts":
        K, N = c["K"], c["N"]
        return {"bytes": A * _weight_bytes(N, K) + (T if c["gather"] else R) * K * SIZE[c["x"]] + R * N * SIZE[c["y"]] +
                4 * (c["E"] + 1) + (4 * R if c["gather"] else 0), "flops": 2 * R * N * K}
    H, I = c["H"], c["I"]
    return {"bytes": A * (2 * _weight_bytes(I, H) + _weight_bytes(H, I)) + T * H * (SIZE[c["x"]] + SIZE[c["y"]]) +
            16 * R + 4 * (c["E"] + 1), "flops": 6 * R * I * H}


def _e4m3(v):
    """v in 64 bits to the nearest e4m3 value: three mantissa bits, ties to even, subnormal step 2^-9."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _codes64(x):
    """Codes and scales of x: the definition's scale, its reciprocal and their product with x are 32-bit values (they
    decide which code a value between two codes takes), so each is rounded to one here as well."""
    M, K = x.shape
    codes = torch.empty(M, K, dtype=torch.float64, device=x.device)
    scales = []
    for b in range(0, K, B):
        t = x[:, b:b + B].double()
        s = torch.clamp(t.abs().max(dim=1, keepdim=True).values / TOP, min=TINY).float().double()
        codes[:, b:b + B] = _e4m3((t * (1.0 / s).float().double()).float().double())
        scales.append(s)
    return codes, torch.cat(scales, dim=1)


def _values64(x):
    codes, s = _codes64(x)
    for j in range(s.shape[1]):
        codes[:, j * B:(j + 1) * B] *= s[:, j:j + 1]
    return codes


def _product64(x, W, S):
    """x [M, K] in 64 bits times the matrix of codes W [N, K] with scales S."""
    y = torch.zeros(x.shape[0], W.shape[0], dtype=torch.float64, device=x.device)
    for n in range(0, W.shape[0], B):
        w = W[n:n + B].double()
        for j in range(S.shape[1]):
            w[:, j * B:(j + 1) * B] *= S[n // B, j].double()
        y[:, n:n + B] = x @ w.t()
    return y


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        return _codes64(s["x"])
    if c["op"] == "f8":
        return _product64(_values64(s["x"]), s["W"], s["S"])
    if c["op"] == "route":
        x = s["x"].double()
        picked = torch.topk(x, c["k"], dim=1).values
        if c["score"] == "softmax":
            w = torch.softmax(picked, 1) if c["norm"] else torch.softmax(x, 1).topk(c["k"], dim=1).values
        else:
            w = torch.sigmoid(picked)
            w = w / w.sum(dim=1, keepdim=True) if c["norm"] else w
        return w, None, None, None, None
    edges = s["offsets"].tolist()
    x = _values64(s["x"])
    if c["op"] == "moe" or c["gather"]:
        x = x[s["rows"].long()]
    parts = []
    for e in range(c["E"]):
        r = x[edges[e]:edges[e + 1]]
        if not len(r):
            continue
        if c["op"] == "experts":
            parts.append(_product64(r, s["W"][e], s["S"][e]))
            continue
        gate = _product64(r, s["Wg"][e], s["Sg"][e])
        h = gate * torch.sigmoid(gate) * _product64(r, s["Wu"][e], s["Su"][e])
        parts.append(_product64(_values64(h.float()), s["Wd"][e], s["Sd"][e]))
    y = torch.cat(parts)
    if c["op"] == "experts":
        return y
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=y.device)
    for j in range(c["k"]):
        out += s["weights"][:, j:j + 1].double() * y[s["slots"][:, j].long()]
    return out
