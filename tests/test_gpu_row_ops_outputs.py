"""RMS norm and SwiGLU with every choice of outputs, on one row per CTA and on CTAs
that stay: the codes, the stream and the rows are the same whichever of them are asked
for, and what is not asked for is not written.

Bounds, u = 2^-24: x_scale 48 u and Xn 49 u and half a step of fp16 (74 u for the sum of
squares at most, half of it under the root, and the roundings beside it), z_scale 12 u;
a SwiGLU code is within half a step of w*127/max|w|, whose error is at most
127 * (12 + 12 + 3) u < 2.1e-4. The norm's codes and the stream are exact."""
import numpy as np
import pytest
import torch

import w8a8_quantized_matmul_b200 as m

pytestmark = pytest.mark.gpu

U, F16 = 2.0 ** -24, 2.0 ** -11
# rows beside an SM's two: 320; columns of 1, 2 and 4 vectors a thread, and either side of 8192
SIZES = [(5, 528), (5, 16400), (320, 240), (320, 528), (330, 4112), (320, 8192), (320, 8208), (300, 16400), (298, 32768)]


def _f64(t):
    return t.cpu().numpy().astype(np.float64)


def _dev(a):
    return None if a is None else torch.from_numpy(a).cuda()


@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("stream", ["none", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", SIZES)
def test_norm(M, K, stream, smooth):
    rng = np.random.default_rng(M + K)
    X = rng.standard_normal((M, K)).astype(np.float16)
    g = (1 + 0.3 * rng.standard_normal(K)).astype(np.float16)
    s = (0.25 + 1.5 * rng.random(K)).astype(np.float32) if smooth else None
    R = None
    if stream != "none":
        R = (3 * rng.standard_normal((M, K))).astype(np.float32 if stream == "fp32" else np.float16)
    h = X.astype(np.float32) if R is None else X.astype(np.float32) + R.astype(np.float32)
    w = h * g.astype(np.float32)
    w = w if s is None else w * s
    codes = np.clip(np.rint(w * np.float32(127) / np.abs(w).max(1, keepdims=True)), -127, 127).astype(np.int8)
    h64 = X.astype(np.float64) if R is None else X.astype(np.float64) + R
    n64 = h64 / np.sqrt((h64 ** 2).mean(1, keepdims=True) + np.float64(np.float32(1e-6))) * g.astype(np.float64)
    scale = np.abs(n64 if s is None else n64 * s).max(1)
    for xn in (None, True):
        for where in (["skip"] if R is None else ["apart", "skip", "in place"]):
            for q in ((True, None) if xn else (True,)):
                r = _dev(R)
                H = {"apart": True, "skip": None, "in place": r}[where]
                Xq, xs, Xn, out = m.int8_rmsnorm_quantize_rows(_dev(X), _dev(g), 1e-6, residual=r, s_rcp=_dev(s), H=H, Xn=xn, Xq=q)
                assert (Xq is None) == (xs is None) == (q is None) and (Xn is None) == (xn is None)
                if q:
                    np.testing.assert_array_equal(Xq.cpu().numpy(), codes)
                    assert (np.abs(_f64(xs) - scale) <= 48 * U * scale).all()
                if xn:
                    assert (np.abs(_f64(Xn) - n64) <= (F16 + 49 * U) * np.abs(n64) + 2.0 ** -25).all()
                if where == "skip":
                    assert out is None and (R is None or np.array_equal(r.cpu().numpy(), R))
                else:
                    assert (out.data_ptr() == r.data_ptr()) == (where == "in place")
                    np.testing.assert_array_equal(out.cpu().numpy(), h.astype(R.dtype))
                    if where == "apart":
                        np.testing.assert_array_equal(r.cpu().numpy(), R)


@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("M,I", SIZES + [(600, 16), (2, 65536)])
def test_swiglu(M, I, smooth):
    rng = np.random.default_rng(M + I)
    GU = (2 * rng.standard_normal((M, 2 * I))).astype(np.float16)
    s = (0.25 + 1.5 * rng.random(I)).astype(np.float32) if smooth else None
    g, up = GU[:, :I].astype(np.float64), GU[:, I:].astype(np.float64)
    z = g / (1 + np.exp(-g)) * up
    w = z if s is None else z * s
    top = np.abs(w).max(1)
    first = None
    for want_z in (None, True):
        for want_q in ((True, None) if want_z else (True,)):
            Zq, zs, Z = m.int8_swiglu_quantize_rows(_dev(GU), s_rcp=_dev(s), Z=want_z, Zq=want_q)
            assert (Zq is None) == (zs is None) == (want_q is None) and (Z is None) == (want_z is None)
            if want_z:
                assert (np.abs(_f64(Z) - z) <= (F16 + 12 * U) * np.abs(z) + 2.0 ** -25).all()
            if want_q:
                assert (np.abs(_f64(zs) - top) <= 12 * U * top).all()
                assert (np.abs(_f64(Zq) - w * 127 / top[:, None]) <= 0.5 + 2.1e-4).all()
                if first is not None:   # the same bits with Z and without
                    assert torch.equal(Zq, first[0]) and torch.equal(zs, first[1])
                first = Zq, zs
