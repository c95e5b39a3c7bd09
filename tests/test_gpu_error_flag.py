"""GPU: the error flag is read after everything that was launched before, on whatever stream."""
import pytest
import torch

import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu


def test_the_flag_waits_for_every_stream():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    x = torch.zeros((128, 64), dtype=torch.bfloat16, device="cuda:0")
    one = torch.ones(1, device="cuda:0")
    streams = [torch.cuda.Stream() for _ in range(3)]   # (made non-blocking)
    torch.cuda.synchronize()
    events = []
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(60_000_000)   # some 30 ms
            h3q.h3q_quantize_nvfp4(x, one)
            events.append(torch.cuda.Event())
            events[-1].record()
    assert h3q.h3q_kernel_error_flag() == 0
    assert all(e.query() for e in events)
