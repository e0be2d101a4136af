"""A paged call that waits for room in the device's queue lets the process's
other threads run."""

import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_other_threads_run_meanwhile():
    import transformer_xl_relative_txl_gb300 as txl

    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    book = dict(table=torch.full((1, 2), -1, dtype=torch.int32, device="cuda"), start=z.clone(), rows=z.clone(),
                refs=torch.zeros(4, dtype=torch.int32, device="cuda"))
    txl.txl_pages_free(book, 16, z)
    torch.cuda.synchronize()
    done, gaps = threading.Event(), [0.0]

    def tick():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    other = threading.Thread(target=tick)
    other.start()
    try:
        # The device is busy for about a second; the queue behind it holds a thousand launches or so.
        torch.cuda._sleep(2_000_000_000)
        longest = 0.0
        for _ in range(4000):
            at = time.perf_counter()
            txl.txl_pages_free(book, 16, z)
            longest = max(longest, time.perf_counter() - at)
    finally:
        done.set()
        other.join()
    assert txl.txl_get_device_status() == 0
    assert longest > 0.3, "no call waited"
    assert max(gaps) < 0.5 * longest
