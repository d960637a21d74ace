"""After a wait that ran out, qmm_device_status() clears the status word and the counters that the launch may have left
behind; a memset of device memory returns before it is done, and streams that do not wait for the default one would run
the next call beside it.  On the CPU: the order of what the library asks of the runtime."""
from host_calls import run


def test_clearing_is_done_before_the_call_returns(tmp_path):
    run(tmp_path, """
for st in (ST, ctypes.c_void_p(0x6000)):
    assert experts(60, 8, 600, 256, st=st) == 0
log()
settle(status=1)
assert L.qmm_device_status(ST) == q.QMM_ETIMEOUT
settle()
events = log()
names = [e[1] for e in events]
sets = [i for i, n in enumerate(names) if n.startswith('memset')]
assert len(sets) == 3, events                       # the status word and two streams' counters
assert 'device-sync' in names[:sets[1]], events     # nothing runs when the counters go
assert names[sets[-1]:].count('device-sync') >= 1, events
""")


def test_an_index_error_is_cleared_before_the_call_returns(tmp_path):
    run(tmp_path, """
assert experts(60, 8, 600, 256) == 0
log()
settle(status=2)
assert L.qmm_device_status(ST) == q.QMM_EINDEX
settle()
names = [e[1] for e in log()]
assert [n for n in names if n.startswith('memset')] == ['memset']
assert names[names.index('memset'):].count('device-sync') >= 1, names
assert L.qmm_device_status(ST) == q.QMM_OK
assert not [e for e in log() if e[1] in ('memset', 'device-sync')]
""")
