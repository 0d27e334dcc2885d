"""The layer grouped by expert (qlinear_prepare_experts, qlinear_grouped_gemm)
against the fp64 product of each row with its expert's packed weights."""
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


def _experts(ql, e, n, k, seed, hadamard=True):
    w = torch.stack([S.weights(n, k, 0.02 * (i % 5 + 1), seed, i) for i in range(e)])
    return ql.qlinear_prepare_experts(w.cuda(), hadamard=hadamard), w


def _tokens(ql, m, k, seed, fmt=None, hadamard=True):
    x = S.activations_fixed_outliers(m, k, max(1, k // 100), 30.0, seed, 1).cuda()
    return ql.qlinear_quantize_act(x, ql.QL_ACT_INT8_F16 if fmt is None else fmt, hadamard=hadamard)


def _offsets(counts, first=0):
    return torch.tensor(np.concatenate(([first], first + np.cumsum(counts))), dtype=torch.int32).cuda()


def _check(ql, q, off, w, y, rows=None, before=0.25, hadamard=True):
    """Each row against its expert's fp64 product, computed on the GPU from the
    oracle-checked packed weights: exact integer-by-6-bit products, so the
    bound is bf16's half step, 2^-8 of the value, and the fp32 sums, at most
    K/16 MMA steps and 64 joins of 2^-22 of the absolute products' sum.  Rows
    outside every segment hold `before`."""
    codes, scales = q["codes"].double(), q["scales"].double()
    n_src, T = codes.shape[0], y.shape[0]
    want = torch.full(y.shape, before, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    rel = (w.K / 16 + 64) * 2.0 ** -22
    off = np.maximum.accumulate([min(max(int(o), 0), T) for o in off.tolist()])
    for e in range(w.E):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi == lo:
            continue
        pw = w.expert(e)
        sf = ql.sf_mma_to_rowmajor(pw.view("sf", torch.uint8, ql.lib.qlinear_sf_bytes(w.N, w.K)).cpu(), w.N, w.K).numpy()
        dense = torch.from_numpy(O.nvfp4_dequantize(pw.view("codes", torch.uint8, w.N * w.K // 2).cpu().numpy()
                                                    .reshape(w.N, -1), sf)).cuda()
        dense *= float(pw.view("gscale", torch.float32, 1).item()) / (128 if hadamard else 1)
        src = torch.arange(lo, hi, device="cuda") if rows is None else rows[lo:hi].long()
        ok = (src >= 0) & (src < n_src)
        a = codes[src.clamp(0, n_src - 1)] * (scales[:n_src][src.clamp(0, n_src - 1)] * ok)[:, None]
        want[lo:hi] = a @ dense.t()
        bound[lo:hi] = want[lo:hi].abs() * 2.0 ** -8 * (1 + rel) + (a.abs() @ dense.abs().t()) * rel * (1 + 2.0 ** -8)
    err = (y.double() - want).abs()
    assert bool(torch.isfinite(err).all())
    bad = (err > bound).nonzero()
    assert bad.numel() == 0, (bad[:4].tolist(), float((err / bound.clamp(min=1e-300)).max()))


def test_prepared_experts_are_the_single_layers(ql):
    for hadamard in (True, False):
        w, raw = _experts(ql, 3, 144, 640, 1, hadamard)
        for e in range(3):
            a, b = w.expert(e), ql.qlinear_prepare_weights(raw[e].cuda(), ql.QL_W_NVFP4, hadamard=hadamard)
            for field, dtype, count in (("codes", torch.uint8, 144 * 320), ("sf", torch.uint8, 256 * 40),
                                        ("gscale", torch.float32, 1)):
                assert torch.equal(a.view(field, dtype, count), b.view(field, dtype, count))
    with pytest.raises(IndexError):
        w.expert(3)


def test_against_the_oracle(ql):
    """Small sizes, row by row, against oracle.decoder_oracle (which the larger
    tests' torch reference restates)."""
    e, n, k = 4, 80, 384
    w, raw = _experts(ql, e, n, k, 2)
    packed = [O.prepare_weights_nvfp4(S.bf16_bits(raw[i])) for i in range(e)]
    q = _tokens(ql, 9, k, 3)
    rows = torch.tensor([3, 3, 8, 0, -1, 2, 9, 1, 1, 1, 5, 6, 7], dtype=torch.int32).cuda()
    off = torch.tensor([1, 4, 4, 9, 11], dtype=torch.int32).cuda()
    y = torch.full((13, n), 0.25, dtype=torch.bfloat16, device="cuda")
    ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, w, rows=rows, Y=y)
    want = D.grouped_product(q["codes"].double().cpu().numpy(), q["scales"].double().cpu().numpy(), rows.tolist(),
                             off.tolist(), packed, True, np.full((13, n), 0.25))
    got = y.double().cpu().numpy()
    # bf16's half step; the fp32 sums of 384 products are off by less than 2^-14 of the largest output
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -14 * np.abs(want).max()).all()
    assert (got[[0, 11, 12]] == 0.25).all() and (got[[4, 6]] == 0).all()
    _check(ql, q, off, w, y, rows)


COUNTS = [
    [1],
    [0, 0, 1, 0],
    [8, 0, 3],
    [5, 9, 17, 0, 1],
    [16, 32, 0, 64],
    [191, 0, 192, 193, 1],
    [0, 700, 0, 0, 33, 0],
    [385, 384, 383, 2, 96],
    [1] * 40,
    [0] * 31 + [7] + [0] * 32 + [20] + [0] * 5,
    [3000, 10],
]


@pytest.mark.parametrize("n,k", [(16, 128), (48, 256), (272, 640), (384, 1920)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_ragged_segments(ql, counts, n, k):
    w, _ = _experts(ql, len(counts), n, k, 4)
    for first, tail, gather in ((0, 0, False), (3, 5, False), (2, 1, True)):
        T = first + sum(counts) + tail
        off = _offsets(counts, first)
        tokens = max(1, T // 2) if gather else T
        q = _tokens(ql, tokens, k, 5 + T)
        rows = None
        if gather:
            rows = torch.randint(0, tokens, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32).cuda()
        y = torch.full((T, n), 0.25, dtype=torch.bfloat16, device="cuda")
        assert ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, w, rows=rows, Y=y) is y
        _check(ql, q, off, w, y, rows)
    assert ql.qlinear_device_status() == 0


@pytest.mark.parametrize("per", [40, 100, 1000])     # rows per expert up to which a tile height is taken
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_ragged_segments_in_tiles(ql, counts, per):
    """The same segments where the call's size asks for tensor-memory tiles of
    each height: experts without rows fill up, rows behind the last segment
    too, and are left as they are."""
    n, k = 1552, 640
    first, T = 3, max(545, sum(counts) + 8)
    counts = counts + [0] * max(0, -(-T // per) - len(counts))
    w, _ = _experts(ql, len(counts), n, k, 24)
    q = _tokens(ql, T // 2, k, 25)
    rows = torch.randint(0, T // 2, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32).cuda()
    y = torch.full((T, n), 0.25, dtype=torch.bfloat16, device="cuda")
    off = _offsets(counts, first)
    ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, w, rows=rows, Y=y)
    _check(ql, q, off, w, y, rows)
    assert ql.qlinear_device_status() == 0


@pytest.mark.parametrize("hadamard", [False, True])
@pytest.mark.parametrize("fmt_name", ["QL_ACT_INT8_F16", "QL_ACT_INT6_F16"])
@pytest.mark.parametrize("tokens", [7, 300])
def test_formats(ql, tokens, fmt_name, hadamard):
    fmt = getattr(ql, fmt_name)
    w, _ = _experts(ql, 3, 160, 512, 6, hadamard)
    q = _tokens(ql, tokens, 512, 7, fmt, hadamard)
    off = _offsets([tokens // 2, 0, tokens - tokens // 2])
    y = ql.qlinear_grouped_gemm(fmt, q, off, w)
    _check(ql, q, off, w, y, hadamard=hadamard)


@pytest.mark.parametrize("total", [12, 900])
def test_offsets_and_rows_out_of_range(ql, total):
    """Offsets beyond the output and descending ones, source rows that do not
    exist: clipped, empty and zero rows, and no other row moves."""
    w, _ = _experts(ql, 4, 64, 256, 8)
    q = _tokens(ql, 10, 256, 9)
    rows = torch.randint(0, 10, (total,), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    rows[::5] = torch.tensor([-1, 10, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64).to(torch.int32).cuda().repeat(total)[
        :rows[::5].numel()]
    for off in ([-5, 3, 3, total // 2, total + 100], [2 ** 31 - 1] * 5, [-2 ** 31] * 5, [0, 0, 0, 0, 2 ** 31 - 1],
                [2, total // 2, 1, 1, 1], [0, total, 0, total, 0]):
        y = torch.full((total, 64), 0.25, dtype=torch.bfloat16, device="cuda")
        o = torch.tensor(off, dtype=torch.int64).to(torch.int32).cuda()
        ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, o, w, rows=rows, Y=y)
        _check(ql, q, o, w, y, rows)
    assert ql.qlinear_device_status() == 0


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts", [[3, 0, 5], [60, 0, 100], [39] * 13, [90] * 6, [200, 150, 250]], ids=len)   # every form
def test_a_bad_row_stays_alone(ql, counts, gather):
    """NaN and infinite codes in rows inside and behind the segments, and in
    row 0, which stands beside the rows that do not exist."""
    w, _ = _experts(ql, len(counts), 2064, 256, 20)
    T = sum(counts) + 6
    q = _tokens(ql, T, 256, 21)
    off = _offsets(counts, 2)
    rows = None
    if gather:
        rows = torch.randint(0, T, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32).cuda()
        rows[3::7] = -1
    y = torch.full((T, 2064), 0.25, dtype=torch.bfloat16, device="cuda")
    want = ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, w, rows=rows, Y=y.clone())
    bad = {key: v.clone() for key, v in q.items() if v is not None}
    hit = torch.tensor([0, 4, 5, T - 1], device="cuda")
    bad["codes"][hit[::2]] = float("nan")
    bad["codes"][hit[1::2], 17] = float("inf")
    got = ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, bad, off, w, rows=rows, Y=y.clone())
    src = torch.arange(T, device="cuda") if rows is None else rows.long()
    keep = ~torch.isin(src, hit)
    assert bool(keep.any()) and torch.equal(got[keep], want[keep])
    if gather:
        inside = torch.arange(T, device="cuda")
        inside = (inside >= 2) & (inside < 2 + sum(counts)) & (src == -1)
        assert bool(inside.any()) and bool((got[inside] == 0).all())


@pytest.mark.parametrize("counts", [[2, 0, 1, 4, 0, 0, 1], [40, 7, 0, 150, 33, 9, 80]])
def test_two_calls_at_once(ql, counts):
    """The same weights on two streams, each call with its own workspace."""
    w, _ = _experts(ql, len(counts), 1920, 640, 22)
    T, off, gen = sum(counts), _offsets(counts), torch.Generator().manual_seed(5)
    qs = [_tokens(ql, 30, 640, 23 + i) for i in range(2)]
    rows = [torch.randint(0, 30, (T,), generator=gen).to(torch.int32).cuda() for _ in range(2)]
    want = [ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, qs[i], off, w, rows=rows[i]) for i in range(2)]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [[ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, qs[i], off, w, rows=rows[i], stream=side[i]) for i in range(2)]
           for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(pair[i], want[i]) for pair in got for i in range(2))
    assert ql.qlinear_device_status() == 0


def test_empty_calls(ql):
    w, _ = _experts(ql, 2, 64, 256, 10)
    q = _tokens(ql, 4, 256, 11)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, _offsets([0, 0]), w, rows=none).shape == (0, 64)
    y = torch.full((4, 64), 0.25, dtype=torch.bfloat16, device="cuda")
    ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, _offsets([0, 0]), w, Y=y)
    assert bool((y == 0.25).all())


@pytest.mark.parametrize("tokens", [6, 500])
def test_a_decoder_block_in_one_graph(ql, tokens):
    """Norm, two expert products with a norm between, replayed with other
    routings and inputs: what the eager calls give, and two graphs at once."""
    e, d, f = 5, 256, 384
    up, _ = _experts(ql, e, f, d, 12)
    down, _ = _experts(ql, e, d, f, 13)
    g1, g2 = (torch.ones(n, dtype=torch.bfloat16, device="cuda") for n in (d, f))
    T = 2 * tokens

    def route(seed):
        gen = torch.Generator().manual_seed(seed)
        ids = torch.randint(0, e, (tokens, 2), generator=gen).flatten()
        order = torch.argsort(ids, stable=True)
        return _offsets(torch.bincount(ids, minlength=e).tolist()), (order // 2).to(torch.int32).cuda()

    def block(x, off, rows, stream=None):
        q = ql.qlinear_norm_quantize(x, g1, ql.QL_ACT_INT8_F16, stream=stream)
        h = ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, up, rows=rows, stream=stream)
        q = ql.qlinear_norm_quantize(h, g2, ql.QL_ACT_INT8_F16, stream=stream)
        return h, ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, down, stream=stream)

    graphs = []
    for i in range(2):
        x = torch.zeros(tokens, d, dtype=torch.bfloat16, device="cuda")
        off, rows = torch.zeros(e + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = block(x, off, rows)
        graphs.append((graph, x, off, rows, outs))
    for step in range(4):
        graph, x, off, rows, outs = graphs[step % 2]
        o, r = route(step)
        x.copy_(S.activations_fixed_outliers(tokens, d, 3, 20.0, step, 1))
        off.copy_(o)
        rows.copy_(r)
        graph.replay()
        want = block(x, o, r)
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = block(x, o, r, side)
    side.synchronize()
    assert torch.equal(got[1], want[1])
    assert ql.qlinear_device_status() == 0
    del graphs


@pytest.mark.parametrize("counts", [[40] * 13, [90] * 6, [200, 150, 250]], ids=len)    # the three tile heights
def test_a_wait_that_runs_out_is_reported(ql, counts):
    w, _ = _experts(ql, len(counts), 2048, 1920, 16)
    q = _tokens(ql, sum(counts), 1920, 17)
    off = _offsets(counts)
    for rows in (None, torch.arange(sum(counts), dtype=torch.int32, device="cuda")):
        want = ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, w, rows=rows)
        torch.cuda.synchronize()
        ql.qlinear_debug_set_wait_limit(0)
        try:
            ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, w, rows=rows)
            torch.cuda.synchronize()
        finally:
            ql.qlinear_debug_set_wait_limit(-1)
        assert ql.qlinear_device_status() == 5 and ql.qlinear_device_status() == 0
        assert torch.equal(ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, w, rows=rows), want)


def test_checkpoint(ql):
    w, _ = _experts(ql, 3, 48, 256, 14)
    q = _tokens(ql, 20, 256, 15)
    off = _offsets([4, 9, 7])
    y = ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, w)
    again = ql.PackedExperts.from_state_dict(w.state_dict(), "cuda")
    w.buf.zero_()
    assert torch.equal(ql.qlinear_grouped_gemm(ql.QL_ACT_INT8_F16, q, off, again), y)
    for e in range(3):
        lo, hi = off[e].item(), off[e + 1].item()
        one = dict(codes=q["codes"][lo:hi].contiguous(), scales=q["scales"][lo:hi].contiguous())
        z = ql.qlinear_gemv(ql.QL_ACT_INT8_F16, one, hi - lo, again.expert(e))
        assert (z - y[lo:hi]).abs().max() <= 2.0 ** -6 * y[lo:hi].abs().max()
