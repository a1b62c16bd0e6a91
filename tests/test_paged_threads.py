"""The paged operators' calls beside other Python threads: a call that waits in a launch lets them run."""
import threading
import time

import pytest
import torch

from tests.test_paged import make_cache, tables

pytestmark = pytest.mark.gpu
STEP = 0.001        # seconds between two looks of the other thread


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls(lib):
    """The operators of the compiled module, each as a call without arguments."""
    c = make_cache(lib, 40, 16, 2, 64, "e4m3", torch.bfloat16, 4)
    q, k, v = (torch.randn(3, h, 64, device="cuda").bfloat16() for h in (8, 2, 2))
    t, lens = tables(3, 5, 20, 3).cuda(), i32([40, 70, 33])
    refs, rows = torch.zeros(50, dtype=torch.int32, device="cuda"), torch.full((3, 5), -1, dtype=torch.int32, device="cuda")
    none, one, a, b = i32([0, 0, 0]), i32([1, 1, 1]), i32([1, 2]), i32([21, 22])
    kept, to = i32([[3, 31, 17]] * 3), i32([[30], [31], [32]])
    return {"append": lambda: lib.sdpa_cache_append(c, k, v, t, lens, q=q),
            "forward": lambda: lib.sdpa_paged_forward(q, c, t, lens, is_causal=True),
            "norm_rotate": lambda: lib.sdpa_norm_rotate(q, k),
            "take": lambda: lib.sdpa_pages_take(refs, rows, none, none, 16),
            "fork": lambda: lib.sdpa_pages_fork(refs, rows, none, none[:1], one[:1], 16),
            "release": lambda: lib.sdpa_pages_release(refs, rows, none, one, 16),
            "copy_pages": lambda: lib.sdpa_cache_copy_pages(c, a, b),
            "compact": lambda: lib.sdpa_cache_compact(c, t, kept, to)}


NAMES = ["append", "forward", "norm_rotate", "take", "fork", "release", "copy_pages", "compact"]


@pytest.mark.parametrize("name", NAMES)
def test_other_threads_run_while_a_launch_waits(sdpa_lib, name):
    """Behind a kernel of about 0.4 s the queue of launches fills up and a call waits for room in it; meanwhile another
    thread looks at the clock every STEP."""
    call = calls(sdpa_lib)[name]
    call()              # (loads the kernel)
    torch.cuda.synchronize()
    looks, stop, spans = [], threading.Event(), []

    def look():
        while not stop.is_set():
            looks.append(time.perf_counter())
            time.sleep(STEP)

    other = threading.Thread(target=look)
    other.start()
    done = torch.cuda.Event()
    try:
        torch.cuda._sleep(700_000_000)
        done.record()
        while len(spans) < 20000 and not done.query():
            start = time.perf_counter()
            call()
            spans.append((start, time.perf_counter()))
    finally:
        stop.set()
        other.join()
        torch.cuda.synchronize()
    start, end = max(spans, key=lambda s: s[1] - s[0])
    if end - start < 100 * STEP:
        pytest.skip("no launch had to wait")
    # (a tenth of the looks that STEP allows: room for a busy machine)
    assert sum(start < x < end for x in looks) >= (end - start) / STEP / 10
