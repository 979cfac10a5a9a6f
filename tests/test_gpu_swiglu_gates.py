"""SwiGLU on rows whose gates are all far below zero, so that the row's scale and
codes come from the exponential's small values, against 64 bits.

Bounds, u = 2^-24: e^g takes ex2 (4 u), the correction's multiply-add (1 u; what the
correction itself is off by is below 2^-40) and no more, whatever the size of g;
|g| t, 1 + t and the last multiply-add 1 u each, the reciprocal 2 u: 10 u. The product
with up and that with s_rcp one more each: 12 u. A code is within half a step of
w*127/max|w|, whose error is at most 127 * (12 + 12 + 3) u < 2.1e-4."""
import numpy as np
import pytest
import torch

import w8a8_quantized_matmul_b200 as m

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("M,I", [(4, 272), (2, 8208), (700, 272), (400, 4112)])
@pytest.mark.parametrize("low,high", [(-10, -1), (-40, -30), (-60, -50), (-85, -30), (-87, -80)])
def test_rows_of_low_gates(M, I, low, high, smooth):
    rng = np.random.default_rng(M + I - low)
    g16 = rng.uniform(low, high, (M, I)).astype(np.float16)
    up16 = (2 * rng.standard_normal((M, I))).astype(np.float16)
    s = (0.25 + 1.5 * rng.random(I)).astype(np.float32) if smooth else None
    GU = torch.from_numpy(np.concatenate([g16, up16], 1)).cuda()
    Zq, zs, _ = m.int8_swiglu_quantize_rows(GU, s_rcp=None if s is None else torch.from_numpy(s).cuda())
    g, up = g16.astype(np.float64), up16.astype(np.float64)
    w = g / (1 + np.exp(-g)) * up * (1.0 if s is None else s)
    top = np.abs(w).max(1)
    assert (np.abs(zs.cpu().numpy().astype(np.float64) - top) <= 12 * U * top).all()
    assert (np.abs(Zq.cpu().numpy() - w * 127 / top[:, None]) <= 0.5 + 2.1e-4).all()


@pytest.mark.parametrize("M", [2, 600])
def test_gates_where_the_exponential_leaves_the_normal_range(M):
    """Below -87.3 silu counts as 0: there it is under 2^-119."""
    GU = torch.full((M, 2 * 48), 3.0, dtype=torch.float16, device="cuda")
    GU[:, :48] = torch.linspace(-65504, -88, 48).half()
    Zq, zs, Z = m.int8_swiglu_quantize_rows(GU, Z=True)
    assert not Zq.any() and not zs.any() and not Z.any()
