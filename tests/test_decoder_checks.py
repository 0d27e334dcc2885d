"""Argument checks of the decoder-block entry points, before anything reaches
a device: the C ABI's status codes and the binding's exceptions."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def ql():
    from bit_quantized_linear_block_b200 import qlinear
    return qlinear


MB = 1 << 20
FAKE = [64 * MB * (i + 1) for i in range(8)]     # far apart, 256-aligned, never dereferenced
INVALID, SHAPE, ALIGN = 1, 2, 3


def test_norm_quantize_c_checks(ql):
    x, r, g, ro, no, codes, sc = FAKE[:7]

    def f(x=x, r=r, g=g, m=4, k=256, eps=1e-6, fmt=ql.QL_ROUTE_INT8, had=1, ro=ro, no=no, codes=codes, sc=sc):
        return ql.lib.qlinear_norm_quantize(x, r, g, m, k, eps, fmt, had, ro, no, codes, sc, None)

    assert f(m=-1) == INVALID and f(m=2 ** 31) == SHAPE
    for k in (0, 100, 32768 + 128, 1 << 21):
        assert f(k=k) == SHAPE
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert f(eps=eps) == INVALID
    for fmt in (ql.QL_ROUTE_NVFP4, ql.QL_ACT_INT8_TENSOR, ql.QL_ACT_NVFP4_DECOMP, ql.QL_ACT_INT6_TENSOR, 99):
        assert f(fmt=fmt) == INVALID
    assert f(fmt=ql.QL_ROUTE_BF16, no=None) == INVALID            # rotated bf16
    assert f(fmt=ql.QL_ROUTE_BF16, had=0) == INVALID              # the norm twice
    assert f(r=None) == INVALID                                   # residual_out without a residual
    for name in ("x", "g", "codes", "sc"):
        assert f(**{name: None}) == INVALID
    for name in ("x", "r", "g", "ro", "no", "codes"):
        assert f(**{name: FAKE[7] + 8}) == ALIGN
    assert f(sc=FAKE[7] + 2) == ALIGN
    assert f(ro=x + 16) == INVALID and f(ro=no) == INVALID        # partial overlap; two outputs in one
    assert f(codes=x) == INVALID and f(codes=g) == INVALID and f(sc=r + 2048 - 4) == INVALID
    assert f(no=codes + 512) == INVALID


def test_norm_quantize_binding_checks(ql):
    x, g = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ql.qlinear_norm_quantize(x, g)
    with pytest.raises(TypeError, match="bfloat16"):
        ql.qlinear_norm_quantize(x.float(), g)
    with pytest.raises(TypeError, match="Tensor"):
        ql.qlinear_norm_quantize(None, g)


def test_gemv_c_checks(ql):
    a, sc, y = FAKE[:3]
    w = ql.Weights(fmt=ql.QL_W_NVFP4, N=1920, K=1920, hadamard=1, codes=FAKE[3], sf=FAKE[4], gscale=FAKE[5])

    def f(fmt=ql.QL_ROUTE_INT8, a=a, sc=sc, m=3, w=w, y=y):
        return ql.lib.qlinear_gemv(fmt, a, sc, m, None if w is None else C.byref(w), y, None)

    assert f(m=-1) == INVALID and f(m=17) == SHAPE and f(w=None) == INVALID
    for fmt in (ql.QL_ROUTE_NVFP4, ql.QL_ACT_INT8_TENSOR, ql.QL_ACT_NVFP4_DECOMP, 99):
        assert f(fmt=fmt) == INVALID
    assert f(a=None) == INVALID and f(y=None) == INVALID and f(sc=None) == INVALID
    assert f(a=a + 8) == ALIGN and f(y=y + 2) == ALIGN and f(sc=sc + 1) == ALIGN
    for change, want in ((dict(K=100), SHAPE), (dict(N=20), SHAPE), (dict(fmt=ql.QL_W_NVFP4_DECOMP), INVALID),
                         (dict(sf=None), INVALID), (dict(codes=None), INVALID)):
        fields = dict(fmt=ql.QL_W_NVFP4, N=1920, K=1920, hadamard=1, codes=FAKE[3], sf=FAKE[4], gscale=FAKE[5])
        assert f(w=ql.Weights(**{**fields, **change})) == want
    q = ql.Weights(fmt=ql.QL_W_QARVD_INT4, N=256, K=256, Kp=288, codes=FAKE[3], gather=FAKE[4], kinfo=FAKE[4],
                   s_norm=FAKE[4], s_out=FAKE[4])
    assert f(w=q) == INVALID


def test_gemv_binding_checks(ql):
    with pytest.raises(TypeError, match="PackedWeights"):
        ql.qlinear_gemv(ql.QL_ROUTE_INT8, {}, 1, object())
    w = ql.PackedWeights(ql.Weights(), torch.zeros(256, dtype=torch.uint8), 16, 128, ql.QL_W_NVFP4)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    for m in (-1, 17):
        with pytest.raises(ValueError, match="0 to 16"):
            ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x), m, w)
    with pytest.raises(ValueError, match="format"):
        ql.qlinear_gemv(ql.QL_ROUTE_NVFP4, dict(codes=x), 1, w)
    with pytest.raises(TypeError, match="int8"):
        ql.qlinear_gemv(ql.QL_ROUTE_INT8, dict(codes=x), 1, w)
    with pytest.raises(ValueError, match="CUDA"):
        ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x), 1, w)
