"""Calls of the 4-bit cache from one thread while another computes: a launch that has to wait for room in the stream's queue
does not keep the interpreter."""
import threading
import time

import pytest

from tests.test_kv4_gpu import pa  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def test_a_waiting_launch_lets_others_run(pa):
    import torch
    rows = torch.randn((1, 1, 64), device="cuda")
    kv, slots = pa.kv4_pool(1, 16, 1, 64), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.paged_attn_append_kv4(rows, rows, slots, kv)
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    longest, done = [0.0], threading.Event()

    def other():
        last = time.perf_counter()
        while not done.is_set():
            now = time.perf_counter()
            longest[0], last = max(longest[0], now - last), now

    t = threading.Thread(target=other)
    t.start()
    time.sleep(0.05)
    began = time.perf_counter()
    torch.cuda._sleep(2_000_000_000)  # a second or so; the queue is full long before
    for _ in range(20000):
        pa.paged_attn_append_kv4(rows, rows, slots, kv)
        if time.perf_counter() - began > 0.6:
            break
    done.set()
    t.join()
    torch.cuda.synchronize()
    assert longest[0] < 0.3, f"the other thread stood still for {longest[0]:.2f} s"
    assert pa.paged_attn_last_error_word() == 0
