"""The products' schedule (mat_mul_gb300/csrc/f8_schedule.h) compiled for the host."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None


def library():
    global _lib
    if _lib is None:
        so = os.path.join(tempfile.mkdtemp(), "f8_schedule.so")
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-ftrapv", "-o", so,
                        os.path.join(HERE, "f8_schedule.cpp")], check=True)
        _lib = ctypes.CDLL(so)
    return _lib


def _p(a):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


def groups(offsets, R, tokens, nb):
    """(tiles before each expert [E + 1], refused groups); offsets None: one matrix."""
    E = 1 if offsets is None else len(offsets) - 1
    cum = np.zeros(E + 1, np.int32)
    off = None if offsets is None else np.ascontiguousarray(offsets, np.int32)
    return cum, library().count_groups(_p(off), E, R, tokens, nb, _p(cum))


def walk(offsets, R, N, K, tokens, cols, G, step, least=4):
    """(pieces [n, 9], plan (tiles, whole, units, sharing)) of a product cut into tiles of `tokens` x `cols`."""
    nb, kb = -(-N // cols), -(-K // 128)
    cum, _ = groups(offsets, R, tokens, nb)
    E = len(cum) - 1
    off = None if offsets is None else np.ascontiguousarray(offsets, np.int32)
    room = int(cum[-1]) * 3 + 2 * G + 16
    out, plan = np.zeros((room, 9), np.int32), np.zeros(4, np.int32)
    n = library().walk(_p(off), _p(cum), E, R, nb, kb, step, least, G, _p(out), room, _p(plan))
    assert n >= 0
    return out[:n], tuple(int(v) for v in plan)


def branch(plan, G):
    """Which rule of the plan: 'few' (every tile among several CTAs), 'shared' (the last rounds over all CTAs), 'whole'."""
    tiles, whole, _, _ = plan
    return "few" if tiles <= G // 2 else "whole" if whole == tiles else "shared"
