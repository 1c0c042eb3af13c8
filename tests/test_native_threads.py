"""The marshalling module lets other Python threads run while the library
works: a launch may wait for a full queue.  (No GPU: the calls are refused.)"""
import sys
import threading
import time

import pytest

import latent_attention_decode_absorbed_b200 as mla
from latent_attention_decode_absorbed_b200 import build as mla_build

CALLS = {"step_plan": 23, "cache_append_slots": 16, "decode_tree": 23, "cache_commit": 16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    mla_build.build()
    return mla.lib()


def _arguments(name):
    """Zeros and None: every call refuses a page size or a count of 0."""
    pointers = {"step_plan": {0, 1, 2, 6, 7, 8, 9, 10, 11, 15, 16, 17, 18, 19, 20, 21},
                "cache_append_slots": {0, 3, 4, 5, 7, 8, 10, 11, 14},
                "decode_tree": {0, 2, 3, 6, 9, 10, 14, 17, 18, 20, 21},
                "cache_commit": {0, 1, 4, 5, 6, 9, 10, 13, 14}}[name]
    args = [None if i in pointers else 0 for i in range(CALLS[name])]
    if name == "cache_append_slots":
        args[2] = -1
    return args


@pytest.mark.parametrize("name", sorted(CALLS))
def test_another_thread_runs_during_a_call(name):
    call, args = getattr(mla.native(), name), _arguments(name)
    assert call(*args) in (mla.MLA_ERR_INVALID_ARG, mla.MLA_ERR_UNSUPPORTED)
    gates, ran = [threading.Lock() for _ in range(8)], []

    def other(gate):
        with gate:
            ran.append(True)

    before = sys.getswitchinterval()
    threads = [threading.Thread(target=other, args=(g,), daemon=True) for g in gates]
    for gate, thread in zip(gates, threads):
        gate.acquire()
        thread.start()
    try:
        sys.setswitchinterval(1000.0)     # only a call that lets go of the interpreter lock lets another thread in
        for gate in gates:
            gate.release()
        end = time.monotonic() + 30       # (a refused call is short: it takes some until a thread that wakes up gets in)
        while not ran and time.monotonic() < end:
            for _ in range(100):
                call(*args)
        seen = bool(ran)
    finally:
        sys.setswitchinterval(before)
    for thread in threads:
        thread.join(10)
    assert seen
