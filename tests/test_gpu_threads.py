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


def test_threads_at_once():
    """Four threads, a stream and a cache of its own each: what one alone gets."""
    H, d, T, P = 2, 64, 40, 16
    table = fa.rope_table(64, d)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    blocks, lens, cu = (torch.tensor(a, dtype=torch.int32, device=DEV) for a in ([[2, 0, 1]], [T], [0, T]))
    slots = blocks[0, pos.long() // P].long() * P + pos % P
    rows = []
    for i in range(4):
        g = torch.Generator().manual_seed(i)
        rows.append([torch.randn(T, h, d, generator=g).to(torch.bfloat16).to(DEV) for h in (H, H, 3 * H)])

    def step(k, v, q, cache):
        fa.cache_append_e2m1(k, v, cache, slots, positions=pos, table=table)
        x = fa.rope(q, pos, table)
        return [x, fa.rope_backward(x, pos, table), *fa.cache_read_e2m1(cache, slots),
                *fa.cache_forward_e2m1(x, cache, blocks, lens, cu)]

    caches = [fa.cache_alloc_e2m1(3, H, P, d) for _ in rows]
    want = [step(*r, c) for r, c in zip(rows, caches)]
    caches = [fa.cache_alloc_e2m1(3, H, P, d) for _ in rows]
    torch.cuda.synchronize()
    wrong, begin = [], threading.Barrier(len(rows))

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            begin.wait(30)
            for n in range(150):
                got = step(*rows[i], caches[i])
                if n % 10 == 0 and not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append((i, n))
            stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(rows))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    fa.check_errors()
    assert not wrong
