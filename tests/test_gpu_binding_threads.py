"""The native binding lets other Python threads run while a launch waits for
room in its stream's queue."""
import threading
import time

import pytest
import torch

from nvfp4_w4a4_quantized_03_b200 import inputs, mq
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


def test_other_threads_run_while_a_launch_waits():
    lin = mq.LinearW4A16(inputs.weight_bf16(64, 64, seed=1).to(dev()))
    x, y = torch.zeros(1, 64, dtype=torch.bfloat16, device=dev()), torch.empty(1, 64, dtype=torch.bfloat16, device=dev())
    lin(x, y)
    torch.cuda.synchronize()
    ticks, done = [], threading.Event()

    def watch():
        while not done.is_set():
            ticks.append(time.perf_counter())
            time.sleep(1e-3)
    t = threading.Thread(target=watch)
    t.start()
    t0 = time.perf_counter()
    torch.cuda._sleep(1_000_000_000)                     # half a second and more
    for _ in range(6000):                                # more than a queue holds
        lin(x, y)
    t1 = time.perf_counter()
    done.set()
    t.join()
    torch.cuda.synchronize()
    assert t1 - t0 > 0.3, t1 - t0                        # the calls did have to wait
    gaps = [b - a for a, b in zip(ticks, ticks[1:])]
    assert max(gaps) < 0.15, max(gaps)
