"""One workspace, allocated for the largest batch, for every batch of a server."""
import pytest
import torch

import w8a8_quantized_matmul_b200 as m

pytestmark = pytest.mark.gpu

N = 72


def _inputs(M, K, n, R, g):
    def rn(*s):
        return torch.randn(*s, device="cuda", generator=g)
    return dict(X=rn(M, K).half(), idx=torch.randint(-1, n, (M,), dtype=torch.int32, device="cuda", generator=g), Y0=rn(M, N).half())


@pytest.mark.parametrize("K,n,R", [(8192, 48, 16), (8192, 4, 64), (4096, 4, 32), (2048, 2, 128)])
def test_smaller_batches_after_the_largest(K, n, R):
    g = torch.Generator(device="cuda").manual_seed(R)
    A = (torch.randn(n, R, K, device="cuda", generator=g) * K ** -0.5).half()
    B = (torch.randn(n, N, R, device="cuda", generator=g) * 0.3).half()
    sc = torch.rand(n, device="cuda", generator=g)
    size = m.int8_adapter_add_workspace_size(1500, N, K, n, R)
    held = torch.full((size + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    for M in (1500, 1025, 1024, 769, 768, 513, 512, 385, 384, 193, 192, 33, 17, 16, 1, 1024, 1500):
        c = _inputs(M, K, n, R, g)
        Y, _ = m.int8_adapter_add(c["X"], A, B, c["idx"], sc, c["Y0"], Y=True, workspace=held[:size])
        own, work = m.int8_adapter_add(c["X"], A, B, c["idx"], sc, c["Y0"], Y=True)
        assert torch.equal(Y, own), M
        assert m.int8_device_status(held) == 0 and work.numel() <= size
    assert bool((held[size:] == 0xA5).all())
