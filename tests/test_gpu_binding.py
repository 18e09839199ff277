"""GPU: the native module's calls beside the program's other Python threads."""
import threading
import time

import pytest
import torch

import chain_synth as cs

pytestmark = pytest.mark.gpu


def test_other_threads_run_while_a_launch_waits():
    # with more launches than the queue holds behind a busy stream, a call waits for the GPU (here about
    # a second); another thread goes on meanwhile
    import chain_gb300 as cg
    q, k = cs.normal((1, 2, 64), 1).cuda(), cs.normal((1, 1, 64), 2).cuda()
    g = torch.ones(64, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    call = lambda: cg.chain_qk_norm_rope(q, k, g, g, None, None, 1e-6, 0, qo, ko)
    call()
    torch.cuda.synchronize()
    stop, gaps = threading.Event(), [0.0]

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps[0] = max(gaps[0], now - last)
            last = now

    t = threading.Thread(target=tick)
    t.start()
    waited = 0.0
    try:
        torch.cuda._sleep(2_000_000_000)
        for _ in range(4000):
            a = time.perf_counter()
            call()
            waited = max(waited, time.perf_counter() - a)
    finally:
        stop.set()
        t.join()
        torch.cuda.synchronize()
    assert waited > 0.3, "no launch had to wait: the queue is longer than the test thinks"
    assert gaps[0] < waited / 2, f"another thread stood still for {gaps[0]:.2f} s of the {waited:.2f} s that a call took"
