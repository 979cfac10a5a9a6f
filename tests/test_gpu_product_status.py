"""A wait that gives up in a product whose caller gave no status word is not lost:
int8_scaled_matmul_status tells of it, once."""
import subprocess
import sys

import pytest
import torch

import w8a8_quantized_matmul_b200 as m
from w8a8_quantized_matmul_b200 import _lib

pytestmark = pytest.mark.gpu


def _case(M, N=512, K=512):
    g = torch.Generator(device="cuda").manual_seed(M)
    Xq = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    Wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    return Xq, torch.rand(M, device="cuda", generator=g), Wq, torch.rand(N, device="cuda", generator=g) * 0.01


@pytest.mark.parametrize("gemm", [False, True])
def test_a_wait_that_gave_up_is_told_once(gemm):
    few, many = _case(4), _case(4000, N=8192)    # the kernel for fewer tokens, and the GEMM
    for c in (few, many):
        m.int8_scaled_matmul(*c)
    assert m.int8_scaled_matmul_status() == _lib.I8MM_OK
    m.selftest_product_status(gemm)
    # products that come after it, with and without a status of their own, leave it there
    own = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = [m.int8_scaled_matmul(*c, status=own) for c in (few, many)]
    got = [m.int8_scaled_matmul(*c) for c in (few, many)]
    assert m.int8_scaled_matmul_status() == _lib.I8MM_ERR_TIMEOUT
    assert m.int8_scaled_matmul_status() == _lib.I8MM_OK
    assert int(own) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_on_a_stream_of_its_own():
    s = torch.cuda.Stream()
    m.selftest_product_status(False, stream=s)
    assert m.int8_scaled_matmul_status(stream=s) == _lib.I8MM_ERR_TIMEOUT
    assert m.int8_scaled_matmul_status() == _lib.I8MM_OK


def test_a_first_call_that_is_captured():
    """Nothing of a first call has to be looked up outside the capture."""
    code = """
import torch, w8a8_quantized_matmul_b200 as m
g = torch.Generator(device="cuda").manual_seed(1)
q = lambda r, c: torch.randint(-127, 128, (r, c), dtype=torch.int8, device="cuda", generator=g)
X, W, x, w = q(M, 512), q(N, 512), torch.ones(M, device="cuda"), torch.ones(N, device="cuda") * 1e-2
Y = torch.empty(M, N, dtype=torch.float16, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    m.int8_scaled_matmul(X, x, W, w, Y=Y)
Y.fill_(7)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(Y, m.int8_scaled_matmul(X, x, W, w)) and m.int8_scaled_matmul_status() == 0
"""
    for M, N in ((4, 512), (4000, 8192)):
        r = subprocess.run([sys.executable, "-c", f"M, N = {M}, {N}\n{code}"], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
