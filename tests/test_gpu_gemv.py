"""The quantized linear layer for few rows (qlinear_gemv) against the fp64
product of the same packed weights, for every operand format."""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as D
from oracle import qlinear_oracle as O
from bit_quantized_linear_block_b200 import synthetic as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bit_quantized_linear_block_b200 import qlinear
    return qlinear


FORMATS = ["QL_ROUTE_INT8", "QL_ACT_INT8_F16", "QL_ROUTE_INT6", "QL_ACT_INT6_F16", "QL_ROUTE_BF16"]


def _layer(ql, n, k, seed, hadamard=True):
    w = S.weights(n, k, 0.02, seed, n + k)
    wq = O.prepare_weights_nvfp4(S.bf16_bits(w), hadamard)
    return ql.qlinear_prepare_weights(w.cuda(), ql.QL_W_NVFP4, hadamard=hadamard), wq


def _operand(ql, x, fmt, hadamard):
    if fmt == ql.QL_ROUTE_BF16:
        return dict(codes=x, scales=None)
    return ql.qlinear_quantize_act(x, fmt, hadamard=hadamard)


def _reference(ql, x, q, fmt, wq, hadamard):
    """The fp64 product r and the bound of each output's error: bf16 output
    rounding (2^-8 of the value); fp32 sums, at most K/16 MMA steps and 64
    joins, each off by at most 2^-22 of the absolute products' sum; for bf16
    rows the f16 rounding of the block-scaled row, 2^-12 of each value (below
    2^-29 of its block's largest: 2^-40 of that largest, under the sums' term)."""
    if fmt == ql.QL_ROUTE_BF16:
        a, scale = O.bf16_bits_to_f32(S.bf16_bits(x.cpu())).astype(np.float64), None
    else:
        a, scale = q["codes"].double().cpu().numpy(), q["scales"].double().cpu().numpy()[:x.shape[0]]
    r = D.nvfp4_product(a, wq, hadamard, scale)
    if scale is None and hadamard:
        a = (a.reshape(-1, 128) @ O.sylvester_hadamard(128).astype(np.float64)).reshape(a.shape)
    absolute = np.abs(a) @ np.abs(O.nvfp4_dequantize(wq["packed"], wq["sb"])).T * float(wq["g"])
    absolute = absolute / (128 if hadamard else 1) * (1 if scale is None else scale[:, None])
    rel = (x.shape[1] / 16 + 64) * 2.0 ** -22 + (2.0 ** -12 if scale is None else 0.0)
    return r, 2.0 ** -8 * np.abs(r) * (1 + rel) + absolute * rel * (1 + 2.0 ** -8)


def _check(ql, x, q, fmt, wq, hadamard, y):
    r, bound = _reference(ql, x, q, fmt, wq, hadamard)
    err = np.abs(y.double().cpu().numpy() - r)
    assert np.isfinite(err).all() and (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())


@pytest.mark.parametrize("fmt_name", FORMATS)
@pytest.mark.parametrize("n,k", [(16, 128), (48, 384), (80, 1152), (272, 640), (1920, 1920), (64, 13824), (5760, 256)])
def test_against_the_product_in_64_bits(ql, n, k, fmt_name):
    fmt = getattr(ql, fmt_name)
    for hadamard in (True, False):
        w, wq = _layer(ql, n, k, 3, hadamard)
        for m in (1, 2, 3, 4, 5, 7, 8, 9, 13, 16):
            x = S.activations_fixed_outliers(m, k, max(1, k // 100), 30.0, m + k, 1).cuda()
            q = _operand(ql, x, fmt, hadamard)
            y = ql.qlinear_gemv(fmt, q, m, w)
            assert y.shape == (m, n) and y.dtype == torch.bfloat16
            _check(ql, x, q, fmt, wq, hadamard, y)
    assert ql.qlinear_device_status() == 0


@pytest.mark.parametrize("m", [1, 6, 16])
def test_agrees_with_the_tiled_product(ql, m):
    """The two forms differ by their fp32 sums' order and one bf16 rounding each."""
    w, wq = _layer(ql, 1920, 1920, 4)
    x = S.activations_fixed_outliers(m, 1920, 8, 50.0, m, 1).cuda()
    q = ql.qlinear_quantize_act(x, ql.QL_ACT_INT8_F16)
    a, b = ql.qlinear_gemv(ql.QL_ACT_INT8_F16, q, m, w), ql.qlinear_gemm(ql.QL_ACT_INT8_F16, q, m, w)
    _, bound = _reference(ql, x, q, ql.QL_ACT_INT8_F16, wq, True)
    assert ((a.double() - b.double()).abs().cpu().numpy() <= 2 * bound).all()


def test_rows_do_not_depend_on_their_company(ql):
    """A row among up to 7 or 15 others, beside a row of NaN, infinity or huge
    values, and repeated: the same bits (the row's products and sums are its
    own).  A single row's sums run in another order: within the bound."""
    w, wq = _layer(ql, 384, 1920, 5)
    x = S.activations_fixed_outliers(8, 1920, 8, 50.0, 9, 1).cuda()
    y = ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x), 8, w)
    assert torch.equal(y, ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x), 8, w))
    for i in range(8):
        one = ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x[i:i + 1].contiguous()), 1, w)
        _check(ql, x[i:i + 1], None, ql.QL_ROUTE_BF16, wq, True, one)
        two = ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x[[i, (i + 1) % 8]].contiguous()), 2, w)
        assert torch.equal(two, y[[i, (i + 1) % 8]])
    both = torch.cat((x, x))
    assert torch.equal(ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=both), 16, w), torch.cat((y, y)))
    bad = x.clone()
    bad[1], bad[4, 5], bad[6, 7] = float("nan"), float("inf"), 3e38
    z = ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=bad), 8, w)
    keep = [0, 2, 3, 5, 7]
    assert torch.equal(y[keep], z[keep])
    zero = torch.zeros_like(x)
    assert bool((ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=zero), 8, w) == 0).all())


def test_values_at_the_ends_of_the_range(ql):
    """bf16 rows of 2^-130 (subnormal) and 2^100: the block scaling keeps them."""
    w, wq = _layer(ql, 64, 256, 6, hadamard=False)
    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    x[0], x[1, 3], x[2] = 2.0 ** -126, 2.0 ** 100, torch.randn(256, generator=torch.manual_seed(0)).bfloat16() * 2.0 ** 60
    y = ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x.cuda()), 3, w)
    r, bound = _reference(ql, x.cuda(), None, ql.QL_ROUTE_BF16, wq, False)
    err = np.abs(y.double().cpu().numpy() - r)
    assert (err[1:] <= bound[1:]).all()
    assert (err[0] <= bound[0] + 2.0 ** -133).all()      # the output is a bf16 subnormal: half a step of 2^-133


def test_empty_and_longer_outputs(ql):
    w, _ = _layer(ql, 48, 128, 7)
    assert ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")), 0,
                           w).shape == (0, 48)
    x = torch.ones(5, 128, dtype=torch.bfloat16, device="cuda")
    y = torch.full((9, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    assert ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x), 5, w, Y=y) is y
    assert bool((y[5:] == 7).all()) and not bool((y[:5] == 7).any())


def test_on_a_side_stream_and_in_a_graph(ql):
    w, _ = _layer(ql, 1920, 1920, 8)
    x = S.activations_fixed_outliers(3, 1920, 8, 50.0, 2, 1).cuda()
    g = torch.ones(1920, dtype=torch.bfloat16, device="cuda")

    def step(inp, stream=None):      # the norm feeds the layer, as in a decoder block
        q = ql.qlinear_norm_quantize(inp, g, ql.QL_ACT_INT8_F16, stream=stream)
        return ql.qlinear_gemv(ql.QL_ACT_INT8_F16, q, 3, w, stream=stream)

    want = step(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(x, side)
    side.synchronize()
    assert torch.equal(got, want)
    graphs, outs, inputs = [], [], []
    for _ in range(2):               # two captured graphs, replayed in turn
        inputs.append(torch.zeros_like(x))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(inputs[-1]))
    for i in (0, 1, 0):
        inputs[i].copy_(x)
        graphs[i].replay()
        assert torch.equal(outs[i], want)
        inputs[i].zero_()
    del graphs


def test_first_calls_inside_a_capture():
    """A process whose first calls of the decoder operators are captured: what
    a launch finds out once must be legal in a capture."""
    code = """
import torch
from bit_quantized_linear_block_b200 import qlinear as ql
x = torch.randn(300, 640, device="cuda").bfloat16()
g = torch.ones(640, device="cuda", dtype=torch.bfloat16)
w = ql.qlinear_prepare_weights((0.02 * torch.randn(1920, 640, device="cuda")).bfloat16())
e = ql.qlinear_prepare_experts((0.02 * torch.randn(3, 1920, 640, device="cuda")).bfloat16())
off = torch.tensor([0, 100, 180, 300], dtype=torch.int32, device="cuda")
few = torch.tensor([0, 1, 1, 5], dtype=torch.int32, device="cuda")
big = torch.randint(0, 300, (900,), device="cuda").to(torch.int32)
off3 = torch.tensor([0, 300, 500, 900], dtype=torch.int32, device="cuda")
def step():
    q = ql.qlinear_norm_quantize(x, g, ql.QL_ACT_INT8_F16, residual=x)
    five = dict(codes=q["codes"][:5], scales=q["scales"][:5])
    return [ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x), 1, w), ql.qlinear_gemv(ql.QL_ACT_INT8_F16, q, 16, w),
            ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, five, few, e), ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, e),
            ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off3, e, rows=big)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and ql.qlinear_device_status() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
