"""An expert layer in 8-bit floats, as a decoder would run it: an 8-bit projection of the tokens (the router's
logits), the router, and the gated MLP of every token's experts; then the same with the grouped product on its
own.  Random weights, quantised here the way a checkpoint holds them (e4m3 codes, one scale per 128 x 128 block).

    python examples/f8_expert_layer.py [tokens] [experts] [choices] [hidden] [intermediate]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mat_mul_gb300 as q  # noqa: E402


def checkpoint(*shape):
    """(codes, scales) of normal weights [..., N, K]."""
    n, k = shape[-2:]
    w = torch.zeros(*shape[:-2], -(-n // 128) * 128, -(-k // 128) * 128, device="cuda")
    w[..., :n, :k] = torch.randn(*shape, device="cuda") / k ** 0.5
    t = w.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))          # [..., n/128, 128, k/128, 128]
    s = t.abs().amax(dim=(-3, -1)) / 448
    codes = (t / s[..., :, None, :, None]).flatten(-2).flatten(-3, -2)
    return codes[..., :n, :k].to(torch.float8_e4m3fn).contiguous(), s.contiguous()


def main(tokens=64, experts=32, choices=4, hidden=2048, intermediate=1024):
    torch.manual_seed(0)
    x = torch.randn(tokens, hidden, device="cuda", dtype=torch.bfloat16)
    Wr, Sr = checkpoint(experts, hidden)
    gate, up, down = (checkpoint(experts, *s) for s in ((intermediate, hidden), (intermediate, hidden),
                                                        (hidden, intermediate)))
    logits = q.qmm_f8(Wr, Sr, x, dtype=torch.float32)
    route = q.qmm_route(logits, choices)
    y = q.qmm_f8_moe(x, route, *gate, *up, *down)

    # the same by hand: one row per (token, choice), in expert order
    g = q.qmm_f8_experts(*gate, x, route.offsets, rows=route.rows, dtype=torch.float32)
    u = q.qmm_f8_experts(*up, x, route.offsets, rows=route.rows, dtype=torch.float32)
    d = q.qmm_f8_experts(*down, torch.nn.functional.silu(g) * u, route.offsets, dtype=torch.float32)
    z = (d[route.slots.long()] * route.weights[:, :, None]).sum(dim=1)
    off = ((y.float() - z).norm() / z.norm()).item()
    if q.qmm_device_status() != q.QMM_OK:
        raise RuntimeError("a kernel reported a timeout or a bad index")
    rows = (route.offsets[1:] - route.offsets[:-1]).tolist()
    print(f"{tokens} tokens, {choices} of {experts} experts each: {min(rows)} to {max(rows)} rows per expert; "
          f"layer against grouped products: relative difference {off:.1e}")
    return off


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:]))
