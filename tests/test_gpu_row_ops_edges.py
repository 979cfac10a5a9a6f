"""SwiGLU and RMS norm on values that are not finite: a row that holds one says so
in its scale, and the rows beside it keep their bits."""
import numpy as np
import pytest
import torch

import w8a8_quantized_matmul_b200 as m

pytestmark = pytest.mark.gpu

INF, NAN = np.inf, np.nan


def _dev(a):
    return None if a is None else torch.from_numpy(a).cuda()


def _silu_up(g, up):
    """The definition in 64 bits: inf for a gate of +inf, NaN for one of -inf (inf/inf)."""
    g, up = np.float64(g), np.float64(up)
    with np.errstate(over="ignore", invalid="ignore"):
        return g / (1 + np.exp(-g)) * up


@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("column", [0, 13, 271])
@pytest.mark.parametrize("M", [3, 600])
@pytest.mark.parametrize("gate,up", [(INF, 2.0), (INF, -3.0), (1.5, INF), (-1.5, INF), (65504, -INF), (INF, INF), (NAN, 1.0), (1.0, NAN),
                                     (-INF, 1.0), (0.0, INF), (INF, 0.0), (-65504, INF)])
def test_swiglu_of_what_is_not_finite(M, column, smooth, gate, up):
    I, row = 272, M - 2
    rng = np.random.default_rng(column)
    GU = (2 * rng.standard_normal((M, 2 * I))).astype(np.float16)
    s = (0.25 + 1.5 * rng.random(I)).astype(np.float32) if smooth else None
    Zq0, zs0, Z0 = m.int8_swiglu_quantize_rows(_dev(GU), s_rcp=_dev(s), Z=True)
    GU[row, column], GU[row, I + column] = gate, up
    Zq, zs, Z = m.int8_swiglu_quantize_rows(_dev(GU), s_rcp=_dev(s), Z=True)
    want = _silu_up(gate, up)
    got = float(Z[row, column])
    assert (np.isnan(got) and np.isnan(want)) or got == want
    scale = float(zs[row])
    assert np.isnan(scale) if np.isnan(want) else scale == INF
    # the row's other values, and the other rows
    rest = torch.ones(M, I, dtype=torch.bool, device="cuda")
    rest[row, column] = False
    assert torch.equal(Z[rest], Z0[rest])
    keep = torch.arange(M, device="cuda") != row
    assert torch.equal(Zq[keep], Zq0[keep]) and torch.equal(zs[keep], zs0[keep])
    # without Z, the same codes and scales
    Zq1, zs1, _ = m.int8_swiglu_quantize_rows(_dev(GU), s_rcp=_dev(s))
    assert torch.equal(Zq1, Zq) and torch.equal(zs1.view(torch.int32), zs.view(torch.int32))


WHERE = [(stream, smooth, where) for stream in ("none", "fp16", "fp32") for smooth in (False, True)
         for where in ("X", "gamma", "residual", "s_rcp")
         if not (where == "residual" and stream == "none") and not (where == "s_rcp" and not smooth)]


@pytest.mark.parametrize("M", [3, 600])
@pytest.mark.parametrize("stream,smooth,where", WHERE)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_norm_of_what_is_not_finite(M, stream, smooth, where, value):
    K, row, column = 528, M - 2, 77
    rng = np.random.default_rng(M)
    a = dict(X=rng.standard_normal((M, K)).astype(np.float16), gamma=(1 + 0.3 * rng.standard_normal(K)).astype(np.float16),
             residual=None, s_rcp=(0.25 + 1.5 * rng.random(K)).astype(np.float32) if smooth else None)
    if stream != "none":
        a["residual"] = (3 * rng.standard_normal((M, K))).astype(np.float16 if stream == "fp16" else np.float32)

    def call():
        return m.int8_rmsnorm_quantize_rows(_dev(a["X"]), _dev(a["gamma"]), residual=_dev(a["residual"]), s_rcp=_dev(a["s_rcp"]))
    q0, s0, _, _ = call()
    of_a_row = where in ("X", "residual")
    a[where][(row, column) if of_a_row else column] = value
    q, s, _, _ = call()
    if of_a_row:
        assert not bool(torch.isfinite(s[row]))
        keep = torch.arange(M, device="cuda") != row
        assert torch.equal(q[keep], q0[keep]) and torch.equal(s[keep], s0[keep])
    else:
        assert not bool(torch.isfinite(s).any())
