"""Products whose tiles are cut and dealt out in every way that the schedule knows, for the tests of the schedule itself
(CPU) and of the kernels (GPU).  SMS is the number of multiprocessors that the rules below are meant for."""
SMS = 152

# (rows, N, K, launches, tokens and columns per tile, CTAs or pairs, step, rule)
def _few(M, N, K, rule, launches=2):
    bt = next(b for b in (16, 32, 64) if b >= min(M, 64))
    return (M, N, K, launches, bt, 128, SMS, 0, rule)


def _pairs(M, N, K, rule):
    return (M, N, K, 2, 256, 256, SMS // 2, 256, rule)


ONE_MATRIX = [
    # weights on the lanes: each tile among several CTAs; rounds of whole tiles; the last rounds shared by all CTAs,
    # with fewer tiles than CTAs, a few more, and two rounds more
    _few(4, 5000, 9216, "few"), _few(33, 1000, 4096, "few"), _few(60, 14336, 4096, "whole"),
    _few(4, 10000, 9216, "shared"), _few(30, 10000, 9216, "shared"), _few(64, 10000, 9216, "shared"),
    _few(4, 19800, 5120, "shared"), _few(20, 19800, 5120, "shared"), _few(3, 39500, 5120, "shared"),
    # x quantised by the product: tiles cut, whole ones in one round and in two
    _few(6, 1024, 5120, "few", 1), _few(8, 14336, 1024, "whole", 1), _few(8, 25600, 512, "whole", 1),
    # tokens on the lanes, pairs of CTAs
    _pairs(300, 2000, 4096, "few"), _pairs(1100, 14336, 1024, "whole"), _pairs(8192, 8192, 128, "whole"),
    _pairs(200, 10300, 9216, "shared"), _pairs(512, 5120, 17408, "shared"), _pairs(1100, 5120, 17408, "shared"),
    _pairs(4096, 5120, 17408, "shared"),
]


# (rows of every expert, N, K, tokens and columns per tile, CTAs, step, rule)
def _groups(sizes, N, K, rule):
    mean = -(-sum(sizes) // len(sizes))
    if mean > 24:
        return (sizes, N, K, 128, 256, SMS, 128, rule)
    return (sizes, N, K, 16 if mean <= 16 else 32, 128, SMS, 0, rule)


EXPERTS = [
    _groups([3, 0, 17, 1, 9, 0, 2, 40], 600, 4096, "few"), _groups([3, 0, 17, 1, 9, 0, 2, 40], 1280, 9216, "whole"),
    _groups([3, 5, 17, 1, 9, 8, 2, 30], 1000, 9216, "shared"), _groups([5, 12, 1, 9, 16], 3900, 5120, "shared"),
    _groups([21] * 8, 1280, 9216, "shared"), _groups([1] * 64, 600, 2048, "whole"),
    _groups([64] + [0] * 63, 1500, 2048, "few"), _groups([0] * 40 + [200] + [0] * 23, 1500, 2048, "whole"),
    _groups([100, 0, 30, 300], 1000, 2048, "few"), _groups([40] * 8, 2560, 9216, "shared"),
    _groups([30, 35, 40, 45, 50], 7900, 5120, "shared"), _groups([100] * 40, 8192, 256, "whole"),
]


# (tokens, choices, experts, H, I, rules of gate and up and of down)
EXPERT_LAYERS = [
    (8, 2, 4, 1152, 1168, "few", "few"), (100, 2, 4, 1152, 1168, "few", "few"),
    (90, 2, 20, 1152, 1168, "whole", "whole"), (400, 2, 20, 1152, 1168, "whole", "whole"),
    (16, 1, 8, 9216, 1280, "shared", "whole"), (240, 1, 8, 9216, 1280, "shared", "whole"),
    (60, 1, 3, 1280, 9216, "whole", "few"), (1000, 4, 40, 256, 2816, "whole", "few"),
]
