"""No write outside the outputs: the decoder-block operators write into the
middle of larger buffers, on ragged shapes, and the margins keep their values;
a run of the operators together, as a block uses them, gives the oracle's
values."""
import numpy as np
import pytest
import torch

from oracle import decoder_oracle as D
from oracle import qlinear_oracle as O
from bit_quantized_linear_block_b200 import synthetic as S

pytestmark = pytest.mark.gpu

BAND = 4096     # elements on each side (16-byte aligned for every type here)


@pytest.fixture(scope="module")
def ql():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bit_quantized_linear_block_b200 import qlinear
    return qlinear


class Guarded:
    """Tensors inside canary margins."""

    def __init__(self):
        self.flats = []

    def make(self, shape, dtype, canary):
        n = int(np.prod(shape))
        flat = torch.full((n + 2 * BAND,), canary, dtype=dtype, device="cuda")
        self.flats.append((flat, n, canary))
        return flat[BAND:BAND + n].view(shape)

    def check(self):
        for flat, n, canary in self.flats:
            assert bool((flat[:BAND] == canary).all()) and bool((flat[BAND + n:] == canary).all())


@pytest.mark.parametrize("m,k", [(1, 128), (3, 384), (5, 1920), (2, 8320), (2, 16512), (150, 1152)])
def test_norm_quantize(ql, m, k):
    for fmt, dtype in ((ql.QL_ROUTE_INT8, torch.int8), (ql.QL_ACT_INT6_F16, torch.float16),
                       (ql.QL_ROUTE_BF16, torch.bfloat16)):
        plain = fmt == ql.QL_ROUTE_BF16
        g = Guarded()
        out = dict(codes=g.make((m, k), dtype, 77), residual=g.make((m, k), torch.bfloat16, 3.0),
                   scales=None if plain else g.make((m,), torch.float32, -5.0),
                   norm=None if plain else g.make((m, k), torch.bfloat16, 9.0))
        x = S.activations_fixed_outliers(m, k, 2, 30.0, m, 1).cuda()
        ql.qlinear_norm_quantize(x, torch.ones(k, dtype=torch.bfloat16, device="cuda"), fmt, hadamard=not plain,
                                 residual=x, keep_norm=not plain, out=out)
        torch.cuda.synchronize()
        g.check()


@pytest.mark.parametrize("m,k", [(3001, 128), (3001, 256), (3001, 512), (3001, 896), (1501, 1920), (3001, 1408), (1001, 4608)])
def test_norm_quantize_many_rows(ql, m, k):
    test_norm_quantize(ql, m, k)


@pytest.mark.parametrize("m", [1, 3, 8, 11, 16])
@pytest.mark.parametrize("n,k", [(16, 128), (112, 256), (144, 1920), (1936, 640)])
def test_gemv(ql, m, n, k):
    w = ql.qlinear_prepare_weights(S.weights(n, k, 0.02, 1, n).cuda(), ql.QL_W_NVFP4)
    x = S.activations_fixed_outliers(m, k, 2, 30.0, m, 1).cuda()
    for fmt in (ql.QL_ROUTE_BF16, ql.QL_ROUTE_INT8, ql.QL_ACT_INT8_F16):
        q = dict(codes=x) if fmt == ql.QL_ROUTE_BF16 else ql.qlinear_quantize_act(x, fmt)
        g = Guarded()
        y = g.make((m, n), torch.bfloat16, 7.0)
        ql.qlinear_gemv(fmt, q, m, w, Y=y)
        torch.cuda.synchronize()
        g.check()
        assert not bool((y == 7.0).all())


@pytest.mark.parametrize("counts", [[1, 0, 2], [3, 1, 15, 0, 2], [33, 0, 65, 7], [70, 129, 0, 90], [193, 400, 31]])
@pytest.mark.parametrize("n,k", [(16, 128), (144, 384), (272, 640)])
def test_grouped_gemm(ql, counts, n, k):
    e, total = len(counts), sum(counts)
    w = ql.qlinear_prepare_experts(torch.stack([S.weights(n, k, 0.02, 1, i) for i in range(e)]).cuda())
    off = torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32).cuda()
    q = ql.qlinear_quantize_act(S.activations_fixed_outliers(total, k, 2, 30.0, 2, 1).cuda(), ql.QL_ACT_INT8_F16)
    for rows in (None, torch.arange(total - 1, -1, -1, dtype=torch.int32, device="cuda")):
        g = Guarded()
        y = g.make((total, n), torch.bfloat16, 7.0)
        ws = None
        need = ql.lib.qlinear_grouped_gemm_ws_bytes(total, ql.C.byref(w.desc), int(rows is not None))
        if need:
            ws = g.make((need,), torch.uint8, 201)
        ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, w, rows=rows, Y=y, ws=ws)
        torch.cuda.synchronize()
        g.check()
    assert ql.qlinear_device_status() == 0


@pytest.mark.parametrize("counts", [[40] * 13, [33, 95, 129, 64, 90, 127], [300, 1, 290]], ids=len)     # the tile heights
def test_grouped_gemm_in_tiles(ql, counts):
    test_grouped_gemm(ql, counts, 2064, 384)


@pytest.mark.parametrize("tokens", [1, 4, 90])
def test_a_block_of_dense_and_expert_layers(ql, tokens):
    """norm -> dense layer (few rows or tiles) -> residual + norm -> two expert
    products with a norm between: each step against the oracle on the step's
    own inputs, so that no step's rounding hides another's."""
    d, f, e, top = 384, 512, 4, 2
    dense_w, up_w, down_w = S.weights(d, d, 0.05, 1, 1), [S.weights(f, d, 0.05, 2, i) for i in range(e)], [
        S.weights(d, f, 0.05, 3, i) for i in range(e)]
    dense = ql.qlinear_prepare_weights(dense_w.cuda(), ql.QL_W_NVFP4)
    up, down = (ql.qlinear_prepare_experts(torch.stack(w).cuda()) for w in (up_w, down_w))
    g = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    gf = torch.ones(f, dtype=torch.bfloat16, device="cuda")
    x = S.activations_fixed_outliers(tokens, d, 3, 20.0, 5, 1).cuda()
    fmt = ql.QL_ACT_INT8_F16

    q = ql.qlinear_norm_quantize(x, g, fmt)
    layer = ql.qlinear_gemv if tokens <= ql.GEMV_MAX_ROWS else ql.qlinear_gemm
    a = layer(fmt, q, tokens, dense)
    q2 = ql.qlinear_norm_quantize(a, g, fmt, residual=x)
    ids = torch.randint(0, e, (tokens * top,), generator=torch.Generator().manual_seed(tokens))
    order = torch.argsort(ids, stable=True)
    off = torch.cat((torch.zeros(1, dtype=torch.long), torch.bincount(ids, minlength=e).cumsum(0))).to(torch.int32).cuda()
    rows = (order // top).to(torch.int32).cuda()
    h = ql.qlinear_grouped_gemm(fmt, q2, off, up, rows=rows)
    q3 = ql.qlinear_norm_quantize(h, gf, fmt)
    y = ql.qlinear_grouped_gemm(fmt, q3, off, down)
    torch.cuda.synchronize()
    assert ql.qlinear_device_status() == 0

    ones = S.bf16_bits(torch.ones(d, dtype=torch.bfloat16)), S.bf16_bits(torch.ones(f, dtype=torch.bfloat16))
    bits = lambda t: S.bf16_bits(t.cpu())                                               # noqa: E731
    f64 = lambda t: t.double().cpu().numpy()                                            # noqa: E731
    for got, res, inp, gamma in ((q, None, x, ones[0]), (q2, bits(x), a, ones[0]), (q3, None, h, ones[1])):
        hh, _, codes, scales = D.norm_quantize(bits(inp), res, gamma, 1e-6, True)
        assert np.array_equal(f64(got["codes"]), codes.astype(np.float64)) and np.array_equal(f64(got["scales"]), scales)
        if res is not None:
            assert np.array_equal(f64(got["residual"]), hh)
    packed = lambda ws: [O.prepare_weights_nvfp4(S.bf16_bits(w)) for w in ws]           # noqa: E731

    def check(got, codes, scales, r, offsets, experts):
        """Within bf16's half step of the fp64 product, and fp32 sums of K
        products in at most K/16 MMA steps and 64 joins, each off by at most
        2^-22 of the absolute products' sum."""
        none = np.zeros(got.shape)
        want = D.grouped_product(codes, scales, r, offsets, experts, True, none)
        positive = [dict(wq, packed=wq["packed"] & 0x77) for wq in experts]              # the E2M1 signs off
        total = D.grouped_product(np.abs(codes), scales, r, offsets, positive, True, none)
        rel = (codes.shape[1] / 16 + 64) * 2.0 ** -22
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) * (1 + rel) + total * rel * (1 + 2.0 ** -8)).all()

    check(f64(a), f64(q["codes"]), f64(q["scales"]), None, [0, tokens], packed([dense_w]))
    check(f64(h), f64(q2["codes"]), f64(q2["scales"]), rows.tolist(), off.tolist(), packed(up_w))
    check(f64(y), f64(q3["codes"]), f64(q3["scales"]), None, off.tolist(), packed(down_w))
