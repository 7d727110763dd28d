"""The native argument marshalling of the per-step calls, as torch and Python
see it (needs a GPU)."""
import threading
import time

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import paged_kv_cache_varlen_gb300 as pkv

from .test_gpu_budget import i32, rope_inputs

pytestmark = pytest.mark.gpu


def test_an_output_made_by_the_call_is_filled_in_deterministic_mode():
    # torch fills memory that nobody has written then; the row of a bad position
    # is such memory
    q, k, v, pool, pos, slots = rope_inputs(5, 4, 2, 64, 3)
    inv = pkv.rope_frequencies(64)[0].cuda()
    pos[3] = -1
    was = torch.are_deterministic_algorithms_enabled()
    junk = torch.ones((5, 4, 64), dtype=torch.bfloat16, device="cuda")
    torch.use_deterministic_algorithms(True)
    try:
        del junk  # (the allocator hands it out again)
        out = pkv.rope_kv_cache_write(q, pool, k, v, i32(pos), i32(slots), inv)
    finally:
        torch.use_deterministic_algorithms(was)
    assert torch.isnan(out[3]).all() and not torch.isnan(out[[0, 1, 2, 4]]).any()


def test_a_dispatch_mode_sees_the_output_made_by_the_call():
    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.names = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.names.append(func.name())
            return func(*args, **(kwargs or {}))

    q, k, v, pool, pos, slots = rope_inputs(5, 4, 2, 64, 3)
    inv, p, s = pkv.rope_frequencies(64)[0].cuda(), i32(pos), i32(slots)
    want = pkv.rope_kv_cache_write(q, pool, k, v, p, s, inv)
    with Seen() as seen:
        out = pkv.rope_kv_cache_write(q, pool, k, v, p, s, inv)
    assert any(n.startswith("aten::empty") for n in seen.names)
    assert torch.equal(out, want)


def test_other_threads_run_while_a_call_waits_for_room_in_the_queue():
    # A launch waits while the stream's queue is full; a call that kept the
    # interpreter lock there would stop every other thread of the program (for
    # good, if the stream waited for one of them).
    q, k, v, pool, pos, slots = rope_inputs(2, 4, 2, 64, 3)
    inv, p, s = pkv.rope_frequencies(64)[0].cuda(), i32(pos), i32(slots)
    out = torch.empty((2, 4, 64), dtype=torch.bfloat16, device="cuda")

    def calls(n):
        for _ in range(n):
            pkv.rope_kv_cache_write(q, pool, k, v, p, s, inv, q_out=out)

    calls(3)
    torch.cuda.synchronize()
    stop, gaps = threading.Event(), []

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    thread = threading.Thread(target=tick)
    thread.start()
    try:
        start = time.perf_counter()
        torch.cuda._sleep(int(1.2e9))  # over half a second at any clock of this GPU
        calls(4000)                    # more than the queue holds
        waited = time.perf_counter() - start
        torch.cuda.synchronize()
    finally:
        stop.set()
        thread.join()
    assert waited > 0.4                # the queue was full
    assert max(gaps) < 0.2
