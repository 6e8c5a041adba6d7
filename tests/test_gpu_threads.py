"""Other Python threads run while a call waits for room in the GPU's queue."""
import threading
import time

import pytest
import torch

import exact_attention_forward_04_gb300 as fa

pytestmark = pytest.mark.gpu

DEV = "cuda"


def calls():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    table, pos = fa.rope_table(16, 64), torch.zeros(4, dtype=torch.int32, device=DEV)
    cache, slots = fa.cache_alloc_e2m1(1, 2, 16, 64), torch.arange(4, device=DEV)
    blocks, lens, cu = (torch.tensor(a, dtype=torch.int32, device=DEV) for a in ([[0]], [4], [0, 4]))
    return {"rope": lambda: fa.rope(x, pos, table), "append": lambda: fa.cache_append_e2m1(x, x, cache, slots),
            "read": lambda: fa.cache_read_e2m1(cache, slots),
            "forward": lambda: fa.cache_forward_e2m1(x, cache, blocks, lens, cu)}


@pytest.mark.parametrize("name", ("rope", "append", "read", "forward"))
def test_a_call_that_waits_holds_no_other_thread(name):
    """Calls behind about a second of other work, until the queue is full and one waits;
    this thread meanwhile wakes up every millisecond."""
    call = calls()[name]
    call()
    torch.cuda.synchronize()
    longest, stream = [0.0], torch.cuda.Stream()

    def many():
        with torch.cuda.stream(stream):
            torch.cuda._sleep(2_000_000_000)
            for _ in range(20000):
                t = time.perf_counter()
                call()
                longest[0] = max(longest[0], time.perf_counter() - t)
                if longest[0] > 0.1:
                    return

    thread = threading.Thread(target=many)
    gap, last = 0.0, time.perf_counter()
    thread.start()
    while thread.is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        gap, last = max(gap, now - last), now
    thread.join()
    torch.cuda.synchronize()
    fa.check_errors()
    assert longest[0] > 0.1, "no call waited: nothing was tested"
    assert gap < longest[0] / 2, f"a call waited {longest[0]:.3f} s, and this thread {gap:.3f} s"
