"""Residual + RMS norm + per-token quantization (qlinear_norm_quantize): the
norm within the roundings of its formula in 64 bits, codes and scales bit for
bit those of the oracle and of qlinear_quantize_act on the norm."""
import numpy as np
import pytest
import torch

from oracle import decoder_oracle as D
from oracle import qlinear_oracle as O
from bit_quantized_linear_block_b200 import synthetic as S

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def ql():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bit_quantized_linear_block_b200 import qlinear
    return qlinear


def _inputs(m, k, seed):
    x = S.activations_fixed_outliers(m, k, max(1, k // 100), 30.0, seed, 1)
    r = S.activations_fixed_outliers(m, k, max(1, k // 100), 10.0, seed, 2)
    g = S.to_bf16(1 + 0.1 * np.random.default_rng(seed).standard_normal(k).astype(np.float32))
    return x, r, g


def _f32(t):
    return t.float().cpu().numpy()


def _check(ql, x, r, g, fmt, hadamard, q, eps=EPS):
    h, y, codes, scales = D.norm_quantize(S.bf16_bits(x), None if r is None else S.bf16_bits(r), S.bf16_bits(g), eps,
                                          hadamard, 31 if fmt in (ql.QL_ROUTE_INT6, ql.QL_ACT_INT6_F16) else 127)
    if r is not None:
        assert np.array_equal(_f32(q["residual"]), h)
    if fmt == ql.QL_ROUTE_BF16:
        assert np.array_equal(_f32(q["codes"]), y)
        return
    assert np.array_equal(_f32(q["codes"]), codes.astype(np.float32))
    assert np.array_equal(_f32(q["scales"])[:len(scales)], scales)
    if q["norm"] is not None:
        assert np.array_equal(_f32(q["norm"]), y)
        again = ql.qlinear_quantize_act(q["norm"], fmt, hadamard=hadamard)
        assert torch.equal(again["codes"], q["codes"]) and torch.equal(again["scales"], q["scales"])


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("fmt_name", ["QL_ROUTE_INT8", "QL_ACT_INT8_F16", "QL_ROUTE_INT6", "QL_ACT_INT6_F16",
                                      "QL_ROUTE_BF16"])
@pytest.mark.parametrize("m,k", [(1, 128), (9, 128), (17, 256), (5, 384), (33, 1920), (3, 5120), (2, 8192), (3, 8320),
                                 (2, 16384), (3, 16512), (2, 32768)])
def test_matches_the_oracle(ql, m, k, fmt_name, residual):
    fmt = getattr(ql, fmt_name)
    x, r, g = _inputs(m, k, m * 7 + k)
    r = r if residual else None
    for hadamard in ((False,) if fmt == ql.QL_ROUTE_BF16 else (False, True)):
        keep = fmt != ql.QL_ROUTE_BF16 and hadamard
        q = ql.qlinear_norm_quantize(x.cuda(), g.cuda(), fmt, hadamard=hadamard,
                                     residual=None if r is None else r.cuda(), eps=EPS, keep_norm=keep)
        torch.cuda.synchronize()
        assert (q["residual"] is None) == (r is None) and (q["norm"] is not None) == keep
        _check(ql, x, r, g, fmt, hadamard, q)
    assert ql.qlinear_device_status() == 0


@pytest.mark.parametrize("fmt_name", ["QL_ROUTE_INT8", "QL_ACT_INT6_F16", "QL_ROUTE_BF16"])
@pytest.mark.parametrize("k", [128, 256, 384, 512, 640, 1152, 1536, 1920, 2304, 4608, 8192, 9216, 13824, 16512])
def test_many_rows_as_few(ql, k, fmt_name):
    """A row's result does not depend on how many rows the call has (the
    rows' split over lanes and warps does): rows of one call against the same
    rows 41 at a time, bit for bit."""
    fmt = getattr(ql, fmt_name)
    m = 3001 if k <= 4608 else 1001
    x, r, g = (t.cuda() for t in _inputs(m, k, 16))
    norm = fmt != ql.QL_ROUTE_BF16
    got = ql.qlinear_norm_quantize(x, g, fmt, residual=r, keep_norm=norm)
    got = {key: v for key, v in got.items() if v is not None}
    assert set(got) == ({"codes", "scales", "residual", "norm"} if norm else {"codes", "residual"})
    for lo in range(0, m, 41):
        part = ql.qlinear_norm_quantize(x[lo:lo + 41], g, fmt, residual=r[lo:lo + 41], keep_norm=norm)
        assert all(torch.equal(v[lo:lo + 41], part[key]) for key, v in got.items())


def test_norm_against_its_formula_in_64_bits(ql):
    m, k = 64, 1920
    x, r, g = _inputs(m, k, 5)
    q = ql.qlinear_norm_quantize(x.cuda(), g.cuda(), ql.QL_ROUTE_BF16, hadamard=False, residual=r.cuda(), eps=EPS)
    h = (x.double() + r.double()).bfloat16().double()   # exact sum of two bf16, one rounding
    y = h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * g.double()
    # rstd, its product with h and the product with gamma each round to fp32
    # (2^-24), y to bf16 (2^-8 of at most one binade's upper end: half a step
    # is 2^-9 of the value's binade, at most 2^-8 of the value)
    err = (q["codes"].double().cpu() - y).abs()
    assert bool((err <= y.abs() * (2.0 ** -8 + 3 * 2.0 ** -24)).all())


def test_rows_that_are_zero_tiny_and_huge(ql):
    k = 640
    x = torch.zeros(5, k, dtype=torch.bfloat16)
    x[1] = 2.0 ** -60                    # the mean vanishes beside eps
    x[2, 7] = 3.0e38                     # squares beyond fp32
    x[3] = S.activations_fixed_outliers(1, k, 3, 50.0, 1, 1)[0]
    x[4] = 1e38
    g = torch.ones(k, dtype=torch.bfloat16)
    for fmt in (ql.QL_ROUTE_INT8, ql.QL_ACT_INT8_F16, ql.QL_ROUTE_BF16):
        q = ql.qlinear_norm_quantize(x.cuda(), g.cuda(), fmt, hadamard=fmt != ql.QL_ROUTE_BF16, eps=EPS)
        _check(ql, x, None, g, fmt, fmt != ql.QL_ROUTE_BF16, q)
        assert bool((q["codes"][0] == 0).all())


def test_a_bad_row_stays_alone(ql):
    m, k = 9, 256
    x, _, g = _inputs(m, k, 3)
    bad = x.clone()
    bad[4, 17], bad[5, 3] = float("nan"), float("inf")
    good = [i for i in range(m) if i not in (4, 5)]
    a = ql.qlinear_norm_quantize(x.cuda(), g.cuda(), ql.QL_ROUTE_INT8, eps=EPS)
    b = ql.qlinear_norm_quantize(bad.cuda(), g.cuda(), ql.QL_ROUTE_INT8, eps=EPS)
    assert torch.equal(a["codes"][good], b["codes"][good]) and torch.equal(a["scales"][good], b["scales"][good])


def test_empty_and_reused_buffers(ql):
    x, r, g = _inputs(6, 1920, 11)
    q = ql.qlinear_norm_quantize(torch.empty(0, 1920, dtype=torch.bfloat16, device="cuda"), g.cuda())
    assert q["codes"].shape == (0, 1920)
    big = dict(codes=torch.full((9, 1920), 77, dtype=torch.int8, device="cuda"),
               scales=torch.full((9,), -1.0, device="cuda"),
               residual=torch.full((9, 1920), 3.0, dtype=torch.bfloat16, device="cuda"),
               norm=torch.full((9, 1920), 3.0, dtype=torch.bfloat16, device="cuda"))
    q = ql.qlinear_norm_quantize(x.cuda(), g.cuda(), ql.QL_ROUTE_INT8, residual=r.cuda(), eps=EPS, keep_norm=True, out=big)
    assert all(q[key] is big[key] for key in big)
    assert bool((big["codes"][6:] == 77).all() and (big["scales"][6:] == -1).all())
    assert bool((big["residual"][6:] == 3).all() and (big["norm"][6:] == 3).all())
    _check(ql, x, r, g, ql.QL_ROUTE_INT8, True, {key: None if key == "norm" else v[:6] for key, v in big.items()})


def test_reused_buffers_of_a_plainer_call(ql):
    """What the earlier result lacks (the sum, the norm) is made."""
    x, r, g = (t.cuda() for t in _inputs(6, 1920, 15))
    want = ql.qlinear_norm_quantize(x, g, ql.QL_ROUTE_INT8, residual=r, keep_norm=True)
    bufs = ql.qlinear_norm_quantize(x, g, ql.QL_ROUTE_INT8)
    q = ql.qlinear_norm_quantize(x, g, ql.QL_ROUTE_INT8, residual=r, keep_norm=True, out=bufs)
    assert q["codes"] is bufs["codes"]
    assert all(torch.equal(q[key], v) for key, v in want.items() if v is not None)


@pytest.mark.parametrize("target", ["X", "residual"])
def test_the_residual_stream_in_place(ql, target):
    x, r, g = _inputs(21, 1920, 12)
    xd, rd = x.cuda(), r.cuda()
    bufs = ql.qlinear_norm_quantize(xd, g.cuda(), ql.QL_ACT_INT8_F16, residual=rd, eps=EPS)
    want = {key: v.clone() for key, v in bufs.items() if v is not None}
    bufs["residual"] = xd if target == "X" else rd
    q = ql.qlinear_norm_quantize(xd, g.cuda(), ql.QL_ACT_INT8_F16, residual=rd, eps=EPS, out=bufs)
    assert all(torch.equal(q[key], want[key]) for key in want)


def test_overlaps_are_refused(ql):
    x, r, g = (t.cuda() for t in _inputs(8, 256, 13))
    flat = torch.zeros(3 * 8 * 256, dtype=torch.bfloat16, device="cuda")
    a, b = flat[:2048].view(8, 256), flat[512:2560].view(8, 256)
    a.copy_(x)
    bufs = ql.qlinear_norm_quantize(x, g, ql.QL_ACT_INT8_F16, residual=r, keep_norm=True)
    for change in (dict(residual=b), dict(codes=a.view(torch.float16)), dict(norm=bufs["residual"])):
        with pytest.raises(ql.QLinearError, match="INVALID_ARG"):
            ql.qlinear_norm_quantize(a, g, ql.QL_ACT_INT8_F16, residual=r, keep_norm=True, out={**bufs, **change})


def test_on_a_side_stream_and_in_a_graph(ql):
    x, r, g = (t.cuda() for t in _inputs(300, 1920, 14))
    want = ql.qlinear_norm_quantize(x, g, ql.QL_ACT_INT8_F16, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ql.qlinear_norm_quantize(x, g, ql.QL_ACT_INT8_F16, residual=r, stream=side)
    side.synchronize()
    assert torch.equal(got["codes"], want["codes"]) and torch.equal(got["scales"], want["scales"])
    graph = torch.cuda.CUDAGraph()
    xin = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        got = ql.qlinear_norm_quantize(xin, g, ql.QL_ACT_INT8_F16, residual=r)
    for _ in range(2):
        xin.copy_(x)
        graph.replay()
        assert torch.equal(got["codes"], want["codes"]) and torch.equal(got["residual"], want["residual"])
        xin.zero_()
    del graph
