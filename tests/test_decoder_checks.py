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


def test_experts_c_checks(ql):
    L = ql.lib
    assert L.qlinear_experts_bytes(4, 1920, 1920) >= 4 * (1920 * 960 + 1920 * 120)
    for e, n, k in ((0, 64, 128), (1025, 64, 128), (4, 20, 128), (4, 64, 100), (1024, 1 << 21, 128)):
        assert L.qlinear_experts_bytes(e, n, k) == 0 and L.qlinear_prepare_experts_ws_bytes(e, n, k) == 0
    desc = ql.Experts()

    def prep(w=FAKE[0], e=4, n=64, k=128, buf=FAKE[1], size=1 << 30, ws=FAKE[2], ws_size=1 << 30):
        return L.qlinear_prepare_experts(w, e, n, k, 1, buf, size, C.byref(desc), ws, ws_size, None)

    assert prep(w=None) == INVALID and prep(buf=None) == INVALID and prep(ws=None) == INVALID
    assert prep(e=0) == SHAPE and prep(n=8) == SHAPE and prep(k=64) == SHAPE
    assert prep(w=FAKE[0] + 8) == ALIGN and prep(buf=FAKE[1] + 16) == ALIGN
    assert prep(size=64) == 6 and prep(ws_size=64) == 6

    good = dict(E=4, N=64, K=128, hadamard=1, codes=FAKE[3], sf=FAKE[4], gscale=FAKE[5])

    def f(fmt=ql.QL_ACT_INT8_F16, a=FAKE[0], sc=FAKE[1], n_a=8, rows=None, off=FAKE[2], t=8, w=good, y=FAKE[6], ws=None,
          ws_bytes=0):
        return L.qlinear_grouped_gemm(fmt, a, sc, n_a, rows, off, t, None if w is None else C.byref(ql.Experts(**w)), y,
                                      ws, ws_bytes, None)

    assert f(t=-1) == INVALID and f(n_a=-1) == INVALID and f(n_a=0) == INVALID and f(w=None) == INVALID
    for name in ("a", "sc", "off", "y"):
        assert f(**{name: None}) == INVALID
    for name in ("codes", "sf", "gscale"):
        assert f(w={**good, name: None}) == INVALID
    for change in (dict(E=0), dict(E=2000), dict(N=24), dict(K=64)):
        assert f(w={**good, **change}) == SHAPE
    for fmt in (ql.QL_ROUTE_INT8, ql.QL_ROUTE_BF16, ql.QL_ROUTE_NVFP4, ql.QL_ACT_INT8_TENSOR, 99):
        assert f(fmt=fmt) == INVALID
    assert f(a=FAKE[0] + 2) == ALIGN and f(y=FAKE[6] + 2) == ALIGN
    need = L.qlinear_grouped_gemm_ws_bytes(1000, C.byref(ql.Experts(**good)), 1)
    assert need == 1000 * 128 * 2 and L.qlinear_grouped_gemm_ws_bytes(1000, C.byref(ql.Experts(**good)), 0) == 0
    assert L.qlinear_grouped_gemm_ws_bytes(8, C.byref(ql.Experts(**good)), 1) == 0      # few rows: no copy
    assert L.qlinear_grouped_gemm_ws_bytes(-1, C.byref(ql.Experts(**good)), 1) == 0
    big = dict(t=1000, rows=FAKE[7])
    assert f(**big) == 6 and f(**big, ws=FAKE[5], ws_bytes=need - 1) == 6 and f(**big, ws=FAKE[5] + 16, ws_bytes=need) == ALIGN
    assert f(off=FAKE[2] + 2) == ALIGN and f(rows=FAKE[7] + 2) == ALIGN and f(sc=FAKE[1] + 2) == ALIGN


def test_experts_binding_checks(ql):
    with pytest.raises(ValueError, match="CUDA"):
        ql.qlinear_prepare_experts(torch.zeros(2, 16, 128, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="PackedExperts"):
        ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, {}, None, object())
    w = ql.PackedExperts(ql.Experts(E=2, N=16, K=128, codes=1 << 20, sf=1 << 20, gscale=1 << 20),
                         torch.zeros(256, dtype=torch.uint8), 2, 16, 128)
    with pytest.raises(ValueError, match="grouped"):
        ql.qlinear_grouped_gemm(ql.QL_ROUTE_INT8, {}, None, w)
    q = dict(codes=torch.zeros(4, 128, dtype=torch.float16), scales=torch.zeros(4))
    with pytest.raises(ValueError, match="CUDA"):
        ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, torch.zeros(3, dtype=torch.int32), w)
    with pytest.raises(IndexError):
        w.expert(2)
    sd = dict(abi=ql.lib.qlinear_abi_version(), sizes=dict(E=2, N=16, K=128, hadamard=1),
              offsets=dict(codes=0, sf=2048, gscale=4096 + 2048), buf=torch.zeros(8192, dtype=torch.uint8))
    ok = ql.PackedExperts.from_state_dict(sd, "cpu")
    assert (ok.E, ok.N, ok.K) == (2, 16, 128) and ok.desc.sf - ok.desc.codes == 2048
    for change in (dict(abi=0), dict(offsets={**sd["offsets"], "gscale": 8192}),
                   dict(offsets={**sd["offsets"], "sf": 100})):
        with pytest.raises(ValueError):
            ql.PackedExperts.from_state_dict({**sd, **change}, "cpu")
