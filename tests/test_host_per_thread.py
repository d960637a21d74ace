"""The per-thread default stream has one handle and a stream of its own in every thread: each gets its own workspace."""
from host_calls import run


def test_every_thread_has_its_own_workspace(tmp_path):
    run(tmp_path, """
per_thread = ctypes.c_void_p(2)                     # cudaStreamPerThread
def work():
    for _ in range(2):
        assert f8(40, 600, 2048, st=per_thread) == 0
for _ in range(3):
    t = threading.Thread(target=work); t.start(); t.join()
events = log()
assert all(e[3] == 2 for e in events if e[1] == 'launch') and len([e for e in events if e[1] == 'launch']) == 12
spaces = [e[3] for e in events if e[1] == 'malloc' and e[4] >= 1 << 21]
assert len(spaces) == len(set(spaces)) == 3, events
counters = [e[3] for e in events if e[1] == 'malloc' and e[4] == 4096]
assert len(counters) == 3
assert L.qmm_release() == 0
assert set(spaces + counters) <= {e[3] for e in log('free')}
""")


def test_the_legacy_default_stream_has_two_names(tmp_path):
    """Null and cudaStreamLegacy are one stream: one workspace, and one lock."""
    run(tmp_path, """
legacy, null = ctypes.c_void_p(1), ctypes.c_void_p(0)
assert moe(50, st=legacy) == 0 and moe(50, st=null) == 0
events = log()
assert len([e for e in events if e[1] == 'malloc' and e[4] >= 1 << 21]) == 1, events
settle(us=2000)
ts = [threading.Thread(target=moe, args=(50,), kwargs={'st': s}) for s in (legacy, null)]
[t.start() for t in ts]; [t.join() for t in ts]
who = [e[0] for e in log('launch')]
assert len(who) == 8 and sum(a != b for a, b in zip(who, who[1:])) == 1, who
""")
