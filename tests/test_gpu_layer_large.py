"""The layer operators on tensors of more than 2^31 elements: the last rows are those of
a call that has them alone, bit for bit."""
import pytest
import torch

import w8a8_quantized_matmul_b200 as m

pytestmark = pytest.mark.gpu

TAIL = 400


def _fill(shape, seed):
    """fp16 rows that repeat every 1000, so that filling them takes no second copy; the last ones of their own."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=torch.float16, device="cuda")
    some = torch.randn(1000, shape[1], device="cuda", generator=g).half()
    for i in range(0, shape[0], 1000):
        t[i:i + 1000] = some[:shape[0] - i]
    t[-TAIL:] = torch.randn(TAIL, shape[1], device="cuda", generator=g).half()
    return t


@pytest.mark.parametrize("stream", ["none", "fp16"])
def test_norm(stream):
    M, K = 66000, 32768
    X, g = _fill((M, K), 1), torch.ones(K, dtype=torch.float16, device="cuda")
    R = X if stream == "fp16" else None
    q, s, n, h = m.int8_rmsnorm_quantize_rows(X, g, residual=R, Xn=True)
    for rows in (slice(0, TAIL), slice(-TAIL, None)):
        q1, s1, n1, h1 = m.int8_rmsnorm_quantize_rows(X[rows], g, residual=None if R is None else R[rows], Xn=True)
        assert torch.equal(q[rows], q1) and torch.equal(s[rows], s1) and torch.equal(n[rows], n1)
        assert R is None or torch.equal(h[rows], h1)


def test_swiglu():
    GU = _fill((35000, 2 * 32768), 2)
    q, s, _ = m.int8_swiglu_quantize_rows(GU)
    for rows in (slice(0, TAIL), slice(-TAIL, None)):
        q1, s1, _ = m.int8_swiglu_quantize_rows(GU[rows])
        assert torch.equal(q[rows], q1) and torch.equal(s[rows], s1)


@pytest.mark.parametrize("N", [4096, 4095])
def test_product(N):
    M, K = 540000, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    Xq = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    Wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    xs, ws = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    Y = m.int8_scaled_matmul(Xq, xs, Wq, ws)
    for rows in (slice(0, TAIL), slice(-TAIL, None)):
        assert torch.equal(Y[rows], m.int8_scaled_matmul(Xq[rows], xs[rows].clone(), Wq, ws))


@pytest.mark.parametrize("N", [4096, 4095])
def test_adapters(N):
    M, K, n, R = 540000, 16, 3, 8
    g = torch.Generator(device="cuda").manual_seed(4)
    X, Y0 = torch.randn(M, K, device="cuda", generator=g).half(), _fill((M, N), 5)
    A = torch.randn(n, R, K, device="cuda", generator=g).half()
    B = torch.randn(n, N, R, device="cuda", generator=g).half()
    idx = torch.randint(-1, n, (M,), dtype=torch.int32, device="cuda", generator=g)
    sc = torch.rand(n, device="cuda", generator=g)
    Y, work = m.int8_adapter_add(X, A, B, idx, sc, Y0, Y=True)
    assert m.int8_device_status(work) == 0
    for rows in (slice(0, TAIL), slice(-TAIL, None)):
        y = Y0[rows].double()
        for a in range(n):
            r = idx[rows] == a
            y[r] += float(sc[a]) * (X[rows][r].double() @ A[a].double().t()) @ B[a].double().t()
        # t and the second sum take at most (K/16 + 40) and (R/8 + 24) steps of fp32, 2^-23 each, of sums
        # of absolute values below 500; the result half a step of fp16
        assert bool(((Y[rows].double() - y).abs() <= y.abs() * 2.0 ** -11 + 70 * 2.0 ** -23 * 500).all())
    assert torch.equal(Y[idx < 0][-TAIL:], Y0[idx < 0][-TAIL:])
