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
