"""The decoder-block operators where their precision, their rules or their
offsets could fail: rotated bf16 rows next to rounding borders and at the ends
of the range, norms too small for their scale, rows beside others, every tile
height of the grouped product, and more than 2^31 elements."""
import numpy as np
import pytest
import torch

from oracle import decoder_oracle as D
from oracle import qlinear_oracle as O
from bit_quantized_linear_block_b200 import synthetic as S
from test_gpu_grouped import COUNTS, _check, _experts, _offsets, _tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ql():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bit_quantized_linear_block_b200 import qlinear
    return qlinear


def _layer(ql, w, hadamard=True):
    return (ql.qlinear_prepare_weights(w.cuda(), ql.QL_W_NVFP4, hadamard=hadamard),
            O.prepare_weights_nvfp4(S.bf16_bits(w), hadamard))


def _bf16_reference(x, wq, hadamard):
    """The fp64 product r of bf16 rows and the bound of each output's error:
    bf16 output rounding, 2^-8 of the value; fp32 sums, K/16 MMA steps for each
    of two terms, K/128 block sums and 64 joins, each off by at most 2^-22 of
    the absolute products' sum; and, when the rows are rotated, for each value
    of a 128-element block two f16 terms (half a step of the second, 2^-23 of
    the value; 2^-39 of the block's largest where that term is a subnormal
    f16) and the rotation's own fp32 sums (one MMA step of 2^-22 and three
    additions of 2^-24 of the block's absolute sum: under 2^-21 of it)."""
    x = O.bf16_bits_to_f32(S.bf16_bits(x.cpu())).astype(np.float64)
    m, k = x.shape
    r = D.nvfp4_product(x, wq, hadamard)
    z, dz = x, np.zeros_like(x)
    if hadamard:
        blocks = x.reshape(m, k // 128, 128)
        z = blocks @ O.sylvester_hadamard(128).astype(np.float64)
        dz = (2.0 ** -23 * np.abs(z) + 2.0 ** -39 * np.abs(z).max(-1, keepdims=True)
              + 2.0 ** -21 * np.abs(blocks).sum(-1, keepdims=True)).reshape(m, k)
        z = z.reshape(m, k)
    w = np.abs(O.nvfp4_dequantize(wq["packed"], wq["sb"])).T * float(wq["g"]) / (128 if hadamard else 1)
    steps = (k / 8 + k / 128 + 64) * 2.0 ** -22
    inner = (np.abs(z) @ w) * steps + (dz @ w) * (1 + steps)
    return r, 2.0 ** -8 * np.abs(r) + inner * (1 + 2.0 ** -8)


def _check_bf16(x, wq, hadamard, y):
    r, bound = _bf16_reference(x, wq, hadamard)
    err = np.abs(y.double().cpu().numpy() - r)
    assert np.isfinite(err).all() and (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())
    return r


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -60, 2.0 ** 90])
@pytest.mark.parametrize("m", [1, 2, 5, 8, 11, 16])
def test_rotated_rows_next_to_f16_borders(ql, m, scale):
    """x = 1.5 at element 0 and 2^-11 at element b rotates to 1.5 + 2^-11 s, s
    the signs of row b of H, every value half an f16 step from 1.5 and rounding
    to it.  A weight row along s has the product 128 * 2^-11, all of it in what
    that rounding drops."""
    at = [1, 2, 3, 5, 7, 8, 16, 31, 32, 33, 64, 65, 96, 100, 126, 127]
    w = torch.zeros(16, 256, dtype=torch.bfloat16)
    w[range(16), at] = 0.5
    w[range(16), [128 + b for b in at]] = 0.5
    w, wq = _layer(ql, w)
    x = torch.zeros(m, 256, dtype=torch.bfloat16)
    for i in range(m):
        x[i, 0], x[i, at[i]] = 1.5 * scale, 2.0 ** -11 * scale
        x[i, 128], x[i, 128 + at[i]] = -3.0 * scale, 2.0 ** -10 * scale
    z = (x[:, :128].double() @ torch.from_numpy(O.sylvester_hadamard(128)).double()).numpy() / scale
    assert (z.astype(np.float16) == 1.5).all()
    y = ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x.cuda()), m, w)
    r = _check_bf16(x, wq, True, y)
    assert (np.abs(r[range(m), range(m)]) > 2.0 ** -11 * scale).all()


@pytest.mark.parametrize("m", [1, 4, 7, 16])
@pytest.mark.parametrize("n,k", [(48, 128), (80, 1152), (64, 13824), (1920, 1920)])
def test_rotated_rows_keep_two_terms(ql, n, k, m):
    w, wq = _layer(ql, S.weights(n, k, 0.02, 31, n + k))
    x = S.activations_fixed_outliers(m, k, max(1, k // 100), 30.0, m + k, 1)
    _check_bf16(x, wq, True, ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x.cuda()), m, w))


@pytest.mark.parametrize("hadamard", [False, True])
@pytest.mark.parametrize("m", [1, 3, 12])
def test_subnormal_rows(ql, m, hadamard):
    """bf16 rows below 2^-126, whole and beside a block of ordinary values:
    weights near 2^60 bring the output back among the normal numbers."""
    n, k = 32, 384
    gen = torch.Generator().manual_seed(m)
    w, wq = _layer(ql, (torch.randn(n, k, generator=gen) * 2.0 ** 60).bfloat16(), hadamard)
    x = (torch.randint(-127, 128, (m, k), generator=gen).double() * 2.0 ** -133).bfloat16()
    x[0] = 2.0 ** -130
    if m > 1:
        x[1, 128:256] = torch.randn(128, generator=gen).bfloat16() * 2.0 ** -120
        x[2, :128] = 0
    y = ql.qlinear_gemv(ql.QL_ROUTE_BF16, dict(codes=x.cuda()), m, w)
    assert bool((y.cpu()[0] != 0).any())
    _check_bf16(x, wq, hadamard, y)


@pytest.mark.parametrize("k", [128, 256, 640, 4608, 16512])
@pytest.mark.parametrize("fmt_name", ["QL_ROUTE_INT8", "QL_ACT_INT8_F16", "QL_ROUTE_INT6", "QL_ACT_INT6_F16"])
def test_rows_whose_norm_is_tiny(ql, fmt_name, k):
    """Rows whose largest magnitude is below qmax / FLT_MAX, so that qmax over it
    is no fp32 number, beside a row of zeros: finite codes of the step 2^-128,
    a subnormal fp32 number (amax / qmax is below it), within half a step of the
    norm as it is returned, and FLT_MAX in place of 2^128 and the product's
    rounding (2^-24 each of at most qmax steps).  fp32 sums of these norms are
    exact: they are multiples of 2^-133 below 2^-120."""
    fmt = getattr(ql, fmt_name)
    qmax = 31 if fmt in (ql.QL_ROUTE_INT6, ql.QL_ACT_INT6_F16) else 127
    gen = torch.Generator().manual_seed(k)
    x = torch.randn(9, k, generator=gen).bfloat16().float()
    x[:, 5::7] = 0
    x[3] = 0
    for hadamard in (False, True):
        gamma = torch.full((k,), 2.0 ** (-131 if hadamard else -127)).bfloat16()
        got = ql.qlinear_norm_quantize(x.bfloat16().cuda(), gamma.cuda(), fmt, hadamard=hadamard, keep_norm=True)
        z = got["norm"].double()
        if hadamard:
            z = (z.view(9, -1, 128) @ torch.from_numpy(O.sylvester_hadamard(128)).double().cuda()).view(9, k)
        amax = z.abs().amax(1)
        assert bool((amax < qmax / 3.4e38).all()) and float(amax[0]) > 0
        codes, scales = got["codes"].double(), got["scales"].double()
        assert bool(torch.isfinite(codes).all()) and float(codes.abs().max()) <= qmax and bool((codes[0] != 0).any())
        assert bool((scales == torch.where(amax > 0, 2.0 ** -128, 0.0)).all()) and bool((codes[3] == 0).all())
        assert bool(((codes * 2.0 ** -128 - z).abs() <= 2.0 ** -128 * (0.5 + 2 * qmax * 2.0 ** -24)).all())


@pytest.mark.parametrize("fmt_name", ["QL_ROUTE_BF16", "QL_ROUTE_INT8", "QL_ACT_INT8_F16"])
@pytest.mark.parametrize("n,k", [(64, 13824), (2560, 1920)])
@pytest.mark.parametrize("m", [2, 3, 6, 8, 9, 16])
def test_rows_among_others_of_one_call_size(ql, m, n, k, fmt_name):
    """For one M a row gives the same bits wherever it stands and whatever the
    other rows hold.  (For another M the sums may run in another order: those
    rows are held to the product in 64 bits.)"""
    fmt = getattr(ql, fmt_name)
    w = ql.qlinear_prepare_weights(S.weights(n, k, 0.02, 32, n).cuda(), ql.QL_W_NVFP4)
    x = S.activations_fixed_outliers(m, k, max(1, k // 100), 30.0, m + k, 1).cuda()
    q = dict(codes=x) if fmt == ql.QL_ROUTE_BF16 else ql.qlinear_quantize_act(x, fmt)
    y = ql.qlinear_gemv(fmt, q, m, w)
    turned = {key: v.roll(1, 0) for key, v in q.items() if v is not None and key in ("codes", "scales")}
    assert torch.equal(ql.qlinear_gemv(fmt, turned, m, w), y.roll(1, 0))
    other = {key: v.clone() for key, v in q.items() if v is not None and key in ("codes", "scales")}
    if fmt == ql.QL_ROUTE_INT8:
        other["codes"][1::2] = 127
        other["scales"][1::2] = float("inf")
    else:
        other["codes"][1::2] = float("nan")
    assert torch.equal(ql.qlinear_gemv(fmt, other, m, w)[::2], y[::2])


# fewest rows per expert that take tensor-memory tiles of this height, where the low tiles do not all run at once
HEIGHTS = {64: 0, 128: 40, 192: 100}


@pytest.mark.parametrize("height", HEIGHTS)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_ragged_segments_at_each_tile_height(ql, counts, height):
    """Every list of segments in a call whose rows, experts and columns ask for
    tiles of this height: rows behind the last segment fill the call up and are
    left as they are."""
    n, k, first = 1552, 640, 3
    counts = counts + [0] * max(0, 6 - len(counts))
    e = len(counts)
    T = max(545, sum(counts) + first + 5, HEIGHTS[height] * e + 1)
    if height != 192:                         # experts without rows keep T / E low
        e = max(e, -(-T // (40 if height == 64 else 100)))
        counts = counts + [0] * (e - len(counts))
    per = T / e
    assert HEIGHTS[height] < per <= {64: 40, 128: 100, 192: T}[height]
    assert (min(e, T) + (T - min(e, T)) // 64) * (-(-n // 128)) > 148
    w, _ = _experts(ql, e, n, k, 33)
    q = _tokens(ql, T // 2, k, 34)
    rows = torch.randint(0, T // 2, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32).cuda()
    off = _offsets(counts, first)
    for r in (rows, None):
        source = q if r is not None else _tokens(ql, T, k, 35)
        y = torch.full((T, n), 0.25, dtype=torch.bfloat16, device="cuda")
        ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, source, off, w, rows=r, Y=y)
        _check(ql, source, off, w, y, r)
    assert ql.qlinear_device_status() == 0


def test_more_than_2_to_31_elements(ql):
    """Inputs, outputs and weights whose element or byte offsets pass 2^31: the
    last rows, columns and experts are those of a small call."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    f16 = ql.QL_ACT_INT8_F16
    m, k = 160000, 13824                                       # norm: 2.2e9 elements
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, k, generator=gen, device="cuda").bfloat16()
    g = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    q, want = ql.qlinear_norm_quantize(x, g, f16), ql.qlinear_norm_quantize(x[-3:].contiguous(), g, f16)
    assert torch.equal(q["codes"][-3:], want["codes"]) and torch.equal(q["scales"][-3:], want["scales"])
    assert bool((q["codes"][:2] == 0).all())
    del x, q

    T, n, k = 290000, 7680, 128                                # rows of Y: 2.2e9 elements
    w, _ = _experts(ql, 2, n, k, 36)
    q = _tokens(ql, 1000, k, 37)
    rows = torch.randint(0, 1000, (T,), generator=gen, device="cuda").to(torch.int32)
    off = torch.tensor([0, 5, T], dtype=torch.int32, device="cuda")
    y = ql.qlinear_grouped_gemm(f16, q, off, w, rows=rows)
    few = torch.tensor([0, 0, 600], dtype=torch.int32, device="cuda")
    assert torch.equal(y[-600:], ql.qlinear_grouped_gemm(f16, q, few, w, rows=rows[-600:].contiguous()))
    assert torch.equal(y[5:605], ql.qlinear_grouped_gemm(f16, q, few, w, rows=rows[5:605].contiguous()))
    del y

    e, n, k = 600, 7680, 1024                                  # experts: 4.7e9 weights, 2.4e9 bytes of codes
    big = torch.zeros(e, n, k, dtype=torch.bfloat16, device="cuda")
    big[-1] = 0.02 * torch.randn(n, k, generator=gen, device="cuda")
    w, last = ql.qlinear_prepare_experts(big), ql.qlinear_prepare_experts(big[-1:].contiguous())
    del big
    for count in (9, 700):                                     # both forms
        q = _tokens(ql, count, k, 38)
        off = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
        off[-1] = count
        y = ql.qlinear_grouped_gemm(f16, q, off, w)
        _check(ql, q, torch.tensor([0, count], dtype=torch.int32, device="cuda"), last, y)
    del w

    n, k = 1 << 17, 32768                                      # a layer: 4.3e9 weights
    block = (0.02 * torch.randn(256, k, generator=gen, device="cuda")).bfloat16()
    w, small = ql.qlinear_prepare_weights(block.repeat(n // 256, 1)), ql.qlinear_prepare_experts(block[None])
    q = _tokens(ql, 3, k, 39)
    y = ql.qlinear_gemv(f16, q, 3, w)
    off = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    for at in (0, 256 * 255, n - 256):
        _check(ql, q, off, small, y[:, at:at + 256].contiguous())
    assert ql.qlinear_device_status() == 0
