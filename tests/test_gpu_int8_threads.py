"""Other Python threads go on while a call of the 8-bit integer experts waits for its launch."""
import ctypes
import threading
import time

import pytest
import torch

from redundant_expert_balancing_amd import _lib as L
from redundant_expert_balancing_amd import int8

from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _addresses():
    return [ctypes.cast(getattr(L.lib(), "moonep_int_" + n), ctypes.c_void_p).value for n in L._INT_CALLS]


def test_a_waiting_call_leaves_other_threads_running():
    """nanosleep in the place of the library's function: its first argument, the shape, is read as
    {int64 seconds, int64 nanoseconds} (R, S and E, K), its second, the rows, as NULL. No
    kernel is launched."""
    say("int threads")
    fast = L._int()
    x = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    q, s = int8.buffers(1, 64)
    wait = L.Shape(0, 0, 200_000_000, 0, 0, 64, 64, L.INFER, L.BF16)
    ticks, stop = [], threading.Event()

    def other():
        while not stop.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.002)
    sleep = ctypes.cast(ctypes.CDLL(None).nanosleep, ctypes.c_void_p).value
    device, stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    good = _addresses()
    thread = threading.Thread(target=other)
    fast.bind((sleep, *good[1:]), device, stream)
    try:
        thread.start()
        time.sleep(0.01)
        begin = time.monotonic()
        assert fast.quantize(wait, 0, 64, x, q, s, None) == 0
        end = time.monotonic()
    finally:
        fast.bind(tuple(good), device, stream)
        stop.set()
        thread.join()
    assert end - begin >= 0.19
    assert sum(begin + 0.02 < t < end - 0.02 for t in ticks) >= 10
    L.moonep_int_quantize(L.Shape(1, 1, 1, 1, 0, 64, 64, L.INFER, L.BF16), 1, 64, x, q, s)
    torch.cuda.synchronize()
    assert not q.any()


def test_two_threads_on_streams_of_their_own():
    """Two layers' products at once, each thread on its own stream and buffers, give what they give
    one after the other."""
    say("int two threads")
    H, Hp, rows = 264, 520, 300
    sh = L.Shape(1, rows, 1, 1, 0, H, Hp, L.INFER, L.BF16)
    gen = torch.Generator("cuda").manual_seed(0)
    w = torch.randn((1, H, Hp), device="cuda", generator=gen).bfloat16()
    wq, ws = int8.weight_buffers(1, H, Hp)
    L.moonep_int_quantize_weight(sh, w, wq, ws)
    jobs = []
    for _ in range(2):
        x = torch.randn((rows, H), device="cuda", generator=gen).bfloat16()
        jobs.append((x, *int8.buffers(rows, H), torch.empty((rows, Hp), device="cuda")))
    want = []
    for x, q, s, c in jobs:
        L.moonep_int_quantize(sh, rows, H, x, q, s)
        L.moonep_int_gemm(sh, rows, q, s, wq, ws, None, c)
        want.append(c.clone())
        q.zero_(), s.zero_(), c.zero_()
    torch.cuda.synchronize()
    errors = []

    def work(job):
        try:
            x, q, s, c = job
            stream = torch.cuda.Stream()
            for _ in range(200):
                L.moonep_int_quantize(sh, rows, H, x, q, s, stream)
                L.moonep_int_gemm(sh, rows, q, s, wq, ws, None, c, stream)
            stream.synchronize()
        except Exception as e:        # reported by the main thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for (_, _, _, c), ref in zip(jobs, want):
        assert torch.equal(c, ref)


def test_a_daemon_thread_waits_in_a_call_while_python_ends():
    """The thread's call returns after the interpreter has begun to go; the process ends as usual."""
    import os
    import subprocess
    import sys
    say("int daemon thread")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import ctypes, sys, threading, time, torch
from redundant_expert_balancing_amd import _lib as L, int8
fast = L._int()
x = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
q, s = int8.buffers(1, 64)
torch.cuda.synchronize()
good = [ctypes.cast(getattr(L.lib(), "moonep_int_" + n), ctypes.c_void_p).value for n in L._INT_CALLS]
sleep = ctypes.cast(ctypes.CDLL(None).nanosleep, ctypes.c_void_p).value
fast.bind((sleep, *good[1:]), torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
wait = L.Shape(0, 0, 500_000_000, 0, 0, 64, 64, L.INFER, L.BF16)
threading.Thread(target=lambda: fast.quantize(wait, 0, 64, x, q, s, None), daemon=True).start()
time.sleep(0.1)
class Last:
    def __del__(self, sleep=time.sleep):
        sleep(1.0)                       # past the end of the call
sys.modules["last"] = Last()
print("at the end", flush=True)
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=60)
    assert done.returncode == 0 and "at the end" in done.stdout, done.stderr
