"""Runs the library's host code in a process of its own over tests/fake_cudart.c, the stand-in for the CUDA runtime:
no GPU, made-up device addresses, a log of what would have been launched."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))

PRELUDE = """
import ctypes, sys, threading
sys.path.insert(0, {root!r})
import mat_mul_gb300 as q
fake = ctypes.CDLL({fake!r})
fake.fake_log.argtypes = [ctypes.c_char_p, ctypes.c_size_t]
fake.fake_log.restype = ctypes.c_size_t
fake.fake_set.argtypes = [ctypes.c_size_t, ctypes.c_int, ctypes.c_int]
L = q.load()
A = 0x100000                      # an address that is aligned and never read
ST = ctypes.c_void_p(0x5000)

def settle(most=1 << 38, status=0, us=0):
    fake.fake_set(most, status, us)

def log(kind=None):
    "The events since the last call: [thread, event, name, first number, second number]."
    buf = ctypes.create_string_buffer(1 << 20)
    out = []
    n = fake.fake_log(buf, len(buf))
    for line in buf.raw[:n].decode().splitlines():
        w = line.split(' ')
        out.append((int(w[0]), w[1], w[2], int(w[3], 16), int(w[4], 16)))
    return [e for e in out if kind is None or e[1] == kind]

def kernels():
    "Every kernel that the library holds."
    buf = ctypes.create_string_buffer(1 << 18)
    fake.fake_kernels.restype = ctypes.c_size_t
    n = fake.fake_kernels(buf, ctypes.c_size_t(len(buf)))
    return buf.raw[:n].decode().split()

def f8(M, N, K, st=ST):
    return L.qmm_f8(A, A, N, K, 2, A, M, K, 2, A, N, st)

def experts(R, E, N, K, rows=True, st=ST):
    return L.qmm_f8_experts(A, A, E, N, K, 2, A, R, K, A, A if rows else None, R, 2, A, N, st)

def route(T, E=64, k=4, st=ST):
    return L.qmm_route(0, A, T, E, E, k, 0, 1, 1.0, A, A, A, A, A, st)

def moe(T, H=256, I=256, E=8, k=2, st=ST):
    return L.qmm_f8_moe(2, A, T, H, H, k, A, A, A, E, I, A, A, A, A, A, A, 2, A, H, st)

def qmm(M, N=2048, K=4096, st=ST, t=q.Q4_K):
    return L.qmm(t, A, N, K, A, M, A, st)

def noalloc(M, N=2048, K=4096, st=ST):
    return L.qmm_noalloc(q.Q4_K, A, N, K, A, M, A, st)

def group(M, N=2048, K=4096, st=ST, n=2):
    arr = lambda t, v: (t * n)(*[v] * n)
    return L.qmm_group(n, arr(ctypes.c_int, q.Q4_K), arr(ctypes.c_void_p, A), arr(ctypes.c_int64, N), K, A, M,
                       arr(ctypes.c_void_p, A), st)

def gate_up(M, N=2048, K=4096, st=ST):
    return L.qmm_gate_up(q.Q4_K, A, q.Q4_K, A, N, K, A, M, A, st)
"""


def run(tmp_path, code):
    """Run `code` after the prelude above; whatever it raises fails the caller."""
    import mat_mul_gb300
    mat_mul_gb300.build()
    fake = str(tmp_path / "fake_cudart.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", fake, os.path.join(HERE, "fake_cudart.c"), "-ldl", "-lpthread"],
                   check=True)
    root = os.path.dirname(HERE)
    r = subprocess.run([sys.executable, "-c", PRELUDE.format(root=root, fake=fake) + code], capture_output=True, text=True,
                       timeout=300, env={**os.environ, "LD_PRELOAD": fake})
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout
