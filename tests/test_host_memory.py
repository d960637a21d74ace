"""What the library does with device memory, on the CPU: refused allocations leave no error behind for the next user of
the runtime, and memory that a captured graph may still use is not freed."""
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


def test_counters_that_a_graph_may_hold_are_kept(tmp_path):
    """qmm_t of more matrices than before needs more counters; a graph captured before holds the address of the old."""
    run(tmp_path, """
assert f8(40, 600, 2048) == 0
small = [e[3] for e in log('malloc') if e[4] == 4096]
assert len(small) == 1
assert L.qmm_t(q.Q8_0, A, 4000, 64, 32, A, 1, A, ST) == 0
events = log()
assert [e for e in events if e[1] == 'malloc' and e[4] == 16384], events
assert small[0] not in [e[3] for e in events if e[1] == 'free'], events
settle(status=1)                                    # both are cleared after a timeout, and freed in the end
assert L.qmm_device_status(ST) == q.QMM_ETIMEOUT
settle()
assert small[0] in [e[3] for e in log('memset')]
assert L.qmm_release() == 0
assert small[0] in [e[3] for e in log('free')]
""")
