"""kda_device_status: one pass over all error words, however many kernels have one."""
import statistics
import threading
import time

import pytest
import torch

import kimi_delta_attention_13_gb300 as kda

pytestmark = pytest.mark.gpu
TIMEOUT, INDEX = 5, 6


def bad_index():
    """A pair out of range in state_copy, then in state_pack: skipped, and recorded."""
    x = torch.zeros(2, 1, 8, 8, device="cuda")
    far = torch.tensor([7], device="cuda")
    kda.state_copy(torch.zeros_like(x), x, far)
    kda.state_pack(torch.zeros(2, 1, 8, 8, device="cuda", dtype=torch.bfloat16), x, far)


def test_all_words_are_cleared_by_one_read():
    assert kda.device_status() == 0
    bad_index()
    assert kda.device_status() == INDEX and kda.device_status() == 0
    bad_index()
    for wait in (kda.diag_device_timeout, kda.diag_linear_timeout, kda.diag_delta_timeout):
        wait(100_000)
        assert kda.device_status() == TIMEOUT      # told before an index
        assert kda.device_status() == 0
    bad_index()
    for wait in (kda.diag_device_timeout, kda.diag_linear_timeout, kda.diag_delta_timeout):
        wait(100_000)
    assert kda.device_status() == TIMEOUT and kda.device_status() == 0


def test_an_error_is_told_once():
    """Reads from several threads, each on a stream of its own."""
    for _ in range(5):
        bad_index()
        torch.cuda.synchronize()
        got, lock = [], threading.Lock()

        def read():
            side = torch.cuda.Stream()
            for _ in range(10):
                code = kda.device_status(stream=side)
                with lock:
                    got.append(code)

        threads = [threading.Thread(target=read) for _ in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        # both words are read in one pass: one reader finds them
        assert sorted(got) == [0] * 39 + [INDEX]


def test_a_read_is_one_copy_and_one_wait():
    """It takes no more than a few times what a kernel and a scalar's way to the host take."""
    x = torch.zeros((), device="cuda")

    def cost(f):
        took = []
        for _ in range(60):
            torch.cuda.synchronize()
            t = time.perf_counter()
            f()
            took.append(time.perf_counter() - t)
        return statistics.median(took[10:])

    scalar = cost(lambda: x.add_(1).item())
    assert cost(kda.device_status) <= 4 * scalar
