"""Calls of several host threads on one stream share its workspace, so the launches of a call have to follow one
another: another thread's launch between a quantiser and its product would hand the product the other call's
activations.  On the CPU: the order of the launches is what is looked at."""
from host_calls import run

CALLS = {
    "f8 of few rows": "f8(40, 600, 2048)",
    "f8 of many rows": "f8(300, 600, 2048)",
    "experts": "experts(60, 8, 600, 256)",
    "router": "route(200)",
    "expert layer": "moe(50)",
    "decode": "qmm(4)",
    "prefill": "qmm(64)",
    "fixed scratch": "noalloc(20)",
    "group, prefill": "group(64)",
    "gate and up": "gate_up(4)",
    "gate and up, prefill": "gate_up(64)",
}


def test_launches_of_a_call_stay_together(tmp_path):
    run(tmp_path, f"calls = {list(CALLS.values())!r}" + """
for c in calls:                   # the buffers have their size before the threads start
    assert eval(c) == 0, (c, L.qmm_last_error())
names, last = {}, None
for c in calls:
    log()
    assert eval(c) == 0
    names[c] = [e[2] for e in log('launch')]
    assert len(names[c]) > 1, c   # (a single launch cannot be parted)
settle(us=100)                    # a launch takes its time, so that threads meet
errors = []
def work(mine):
    for i in range(12):
        c = calls[(i * 5 + mine) % len(calls)]
        if eval(c) != 0: errors.append(c)
ts = [threading.Thread(target=work, args=(m,)) for m in range(4)]
[t.start() for t in ts]; [t.join() for t in ts]
assert not errors, errors
got = log('launch')
at = 0
while at < len(got):              # every run of launches by one thread is one whole call
    fits = [c for c in calls if [e[2] for e in got[at:at + len(names[c])]] == names[c] and
            len({e[0] for e in got[at:at + len(names[c])]}) == 1]
    assert fits, (at, got[at:at + 4])
    at += max(len(names[c]) for c in fits)
assert len({e[0] for e in got}) == 4
""")


def test_calls_on_different_streams_do_not_wait_for_one_another(tmp_path):
    run(tmp_path, """
other = ctypes.c_void_p(0x6000)
for st in (ST, other): assert moe(50, st=st) == 0
log()
settle(us=20000)                  # four launches: 80 ms a call
def work(st): moe(50, st=st)
ts = [threading.Thread(target=work, args=(s,)) for s in (ST, other)]
[t.start() for t in ts]; [t.join() for t in ts]
who = [e[0] for e in log('launch')]
assert len(who) == 8 and sum(a != b for a, b in zip(who, who[1:])) > 1, who
""")


def test_no_call_holds_the_lock_after_it_returns(tmp_path):
    """Refused, failed and nested calls too: another thread gets through after each."""
    run(tmp_path, """
def through():
    done = []
    t = threading.Thread(target=lambda: done.append(moe(50)), daemon=True)
    t.start(); t.join(20)
    assert done == [0], done
for call, rc in ((lambda: f8(40, 600, 24), q.QMM_EINVAL_SHAPE), (lambda: gate_up(64), 0), (lambda: qmm(1), 0),
                 (lambda: L.qmm_release(), 0), (lambda: L.qmm_device_status(ST), 0)):
    assert call() == rc
    through()
settle(most=1 << 20)
assert moe(3000, st=ctypes.c_void_p(0x9000)) == q.QMM_ENOMEM
settle()
through()
settle(status=1)
assert L.qmm_device_status(ST) == q.QMM_ETIMEOUT
settle()
through()
""")
