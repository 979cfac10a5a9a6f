"""The bounded wait that the kernels' roles share: after one that gave up, the next
gives up at once instead of waiting its own two seconds."""
import time

import pytest
import torch

import w8a8_quantized_matmul_b200 as m
from w8a8_quantized_matmul_b200 import _lib

pytestmark = pytest.mark.gpu


def test_a_second_wait_gives_up_at_once():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert m.selftest_wait_timeout() == _lib.I8MM_ERR_TIMEOUT
    torch.cuda.synchronize()
    assert 1.9 < time.perf_counter() - t0 < 3.5
    # the context goes on
    assert int(status + 1) == 1
