"""Every kernel of the 8-bit-float operators is reached by some call.  On the CPU: the library's own list of its kernels
against what a sweep of calls launches."""
from host_calls import run


def test_no_kernel_is_out_of_reach(tmp_path):
    run(tmp_path, """
for t in range(3):                                  # value types; whole groups of 8, of 4, neither
    for K, ld in ((256, 256), (260, 260), (256, 260), (255, 255), (256, 257)):
        assert L.qmm_f8_quantize(t, A, 4, K, ld, A, A, ST) == 0
for M in (1, 4, 13, 16, 20, 33, 64, 65, 128, 200, 300, 1000, 5000):
    for N, K in ((128, 128), (1024, 5120), (5120, 5120), (14336, 4096)):
        assert f8(M, N, K) == 0
for E in (1, 4, 64):
    for R in (1, 40, 20 * E, 300, 900, 5000):
        assert experts(R, E, 600, 1024) == 0
        for t in range(3):
            assert L.qmm_f8_moe(t, A, R, 256, 256, 1, A, A, A, E, 256, A, A, A, A, A, A, t, A, 256, ST) == 0
for T in (5, 200, 20000):
    for E in (8, 60, 100, 200, 400, 1000):
        assert route(T, E) == 0
launched = {e[2] for e in log('launch')}
mine = {k for k in kernels() if 'f8_' in k or 'route_' in k}
assert len(mine) > 20 and launched <= set(kernels())
assert mine == launched, sorted(mine - launched)
""")
