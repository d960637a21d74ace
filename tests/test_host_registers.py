"""The product for many rows splits the registers of a block between its warps, which needs what the launch brings: a
build that gave the kernel fewer would wait for them forever.  Such a build runs those products on the other kernel.  On
the CPU: what is launched for the register counts that a stand-in reports."""
from host_calls import run


def test_products_run_whatever_the_compiler_gave(tmp_path):
    run(tmp_path, """
calls = [lambda: f8(300, 600, 2048), lambda: f8(5000, 5120, 5120), lambda: experts(900, 4, 600, 1024),
         lambda: moe(900)]
def names(call):
    log()
    assert call() == 0, L.qmm_last_error()
    return [e[2] for e in log('launch')]
fake.fake_registers(64)                             # too few for any split
few = [names(c) for c in calls]
assert not any('f8_wide' in n for ns in few for n in ns), few
fake.fake_registers(0)                              # what the build has
have = [names(c) for c in calls]
assert all(any('f8_wide' in n for n in ns) for ns in have), have
assert [len(a) for a in few] == [len(a) for a in have]
""")


def test_more_registers_than_the_split_needs(tmp_path):
    run(tmp_path, """
fake.fake_registers(168)                            # 96 are enough for the gated pair
assert moe(900) == 0 and f8(300, 600, 2048) == 0
assert sum('f8_wide' in e[2] for e in log('launch')) == 3
""")
