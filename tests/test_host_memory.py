"""What the library does with device memory, on the CPU: refused allocations leave no error behind for the next user of
the runtime."""
from host_calls import run


def test_a_refused_allocation_leaves_no_error_behind(tmp_path):
    """The runtime keeps the error of a failed call until somebody asks for it: PyTorch would ask after its next launch,
    and raise."""
    run(tmp_path, """
for call in (lambda: moe(3000), lambda: experts(3000, 8, 600, 4096), lambda: f8(3000, 600, 4096),
             lambda: route(200000), lambda: qmm(3000), lambda: gate_up(3000)):
    assert L.qmm_release() == 0
    assert route(4) == 0
    settle(most=1 << 16)
    rc = call()
    settle()
    assert rc == q.QMM_ENOMEM, rc
    assert b'out of memory' in L.qmm_last_error()
    assert fake.fake_last_error() == 0
    assert call() == 0
""")
