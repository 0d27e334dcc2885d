"""Pins of oracle/decoder_oracle.py: the bf16 rounding against torch's, the
norm in closed form and against torch in fp64, the product against exact
rational arithmetic and the other oracle's products, and the grouped product
against the rows' own."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import decoder_oracle as D
from oracle import qlinear_oracle as O
from bit_quantized_linear_block_b200 import synthetic as S


def test_bf16_rounding_is_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000), rng.standard_normal(4000) * 1e-38, [0.0, -0.0, 3e38, -3e38]])
    x = x.astype(np.float32)
    ties = (x[:4000].view(np.uint32) & 0xFFFF0000 | 0x8000).view(np.float32)
    for v in (x, ties):
        assert np.array_equal(D.f32_to_bf16(v).view(np.uint32),
                              torch.from_numpy(v).bfloat16().float().numpy().view(np.uint32))


def test_norm_in_closed_form():
    k = 256
    x = S.to_bf16(np.stack([np.full(k, 3.0), np.zeros(k), np.tile([4.0, -4.0], k // 2)]))
    g = S.to_bf16(np.full(k, 2.0))
    h, y = D.rms_norm(S.bf16_bits(x), None, S.bf16_bits(g), 1e-12)
    assert np.array_equal(h, x.float().numpy())
    assert (y[0] == 2.0).all() and (y[1] == 0).all() and (y[2] == np.tile([2.0, -2.0], k // 2)).all()
    _, y = D.rms_norm(S.bf16_bits(x), None, S.bf16_bits(g), 7.0)       # 3 / sqrt(9 + 7) * 2
    assert (y[0] == 1.5).all()
    h, _ = D.rms_norm(S.bf16_bits(x), S.bf16_bits(x), S.bf16_bits(g), 1.0)
    assert np.array_equal(h, 2 * x.float().numpy())


def test_norm_against_torch_in_fp64():
    x, r = (S.activations_fixed_outliers(7, 640, 6, 30.0, s, 1) for s in (1, 2))
    g = S.to_bf16(1 + 0.1 * np.random.default_rng(3).standard_normal(640).astype(np.float32))
    h, y = D.rms_norm(S.bf16_bits(x), S.bf16_bits(r), S.bf16_bits(g), 1e-5)
    h64 = (x.double() + r.double()).bfloat16().double()
    want = h64 / (h64.square().mean(1, keepdim=True) + 1e-5).sqrt() * g.double()
    assert np.array_equal(h, h64.float().numpy())
    # three fp32 roundings (2^-24 each) and bf16's half step (2^-8 of the value)
    assert (np.abs(y - want.numpy()) <= np.abs(want.numpy()) * (2.0 ** -8 + 4 * 2.0 ** -24)).all()


@pytest.mark.parametrize("qmax", [127, 31])
def test_codes_are_the_token_quantizers(qmax):
    x = S.activations_fixed_outliers(5, 256, 3, 30.0, 4, 1)
    g = S.to_bf16(np.ones(256))
    h, y, q, s = D.norm_quantize(S.bf16_bits(x), None, S.bf16_bits(g), 1e-6, True, qmax)
    q2, s2 = O.int8_per_token(O.block_hadamard(y), qmax)
    assert np.array_equal(q, q2) and np.array_equal(s, s2) and np.abs(q).max() == qmax
    q3, _ = O.int8_per_token(y, qmax)
    assert np.array_equal(D.norm_quantize(S.bf16_bits(x), None, S.bf16_bits(g), 1e-6, False, qmax)[2], q3)


def test_product_in_exact_arithmetic():
    rng = np.random.default_rng(5)
    w = S.weights(16, 128, 0.02, 6, 1)
    for hadamard in (False, True):
        wq = O.prepare_weights_nvfp4(S.bf16_bits(w), hadamard)
        dense = O.nvfp4_dequantize(wq["packed"], wq["sb"])
        a = rng.integers(-127, 128, (2, 128))
        s = np.array([0.5, 0.125])
        y = D.nvfp4_product(a, wq, hadamard, s)
        for m in range(2):
            for n in (0, 7, 15):
                exact = sum(Fraction(int(a[m, k])) * Fraction(float(dense[n, k])) for k in range(128))
                exact *= Fraction(float(wq["g"])) * Fraction(float(s[m])) / (128 if hadamard else 1)
                assert abs(Fraction(float(y[m, n])) - exact) <= abs(exact) * Fraction(1, 2 ** 50) + Fraction(1, 2 ** 80)
    # unquantized rows: rotating both sides leaves the product of the weights' own rotation
    x = rng.standard_normal((3, 128))
    wq = O.prepare_weights_nvfp4(S.bf16_bits(w), True)
    unrotated = O.nvfp4_dequantize(wq["packed"], wq["sb"]) @ O.sylvester_hadamard(128) / 128
    assert np.allclose(D.nvfp4_product(x, wq, True), x @ unrotated.T * float(wq["g"]), rtol=1e-12, atol=1e-14)


def test_grouped_rows_are_the_experts_products():
    packed = [O.prepare_weights_nvfp4(S.bf16_bits(S.weights(16, 128, 0.02, 7, e))) for e in range(3)]
    codes = np.random.default_rng(8).integers(-127, 128, (4, 128)).astype(np.float64)
    scales = np.array([1.0, 0.5, 0.25, 2.0])
    before = np.full((8, 16), 9.0)
    rows = [0, 2, 2, 3, 4, -1, 1, 0]
    y = D.grouped_product(codes, scales, rows, [1, 3, 3, 7], packed, True, before)
    assert (y[0] == 9).all() and (y[7] == 9).all() and (y[4] == 0).all() and (y[5] == 0).all()
    for r, e in ((1, 0), (2, 0), (3, 2), (6, 2)):
        assert np.array_equal(y[r], D.nvfp4_product(codes, packed[e], True, scales)[rows[r]])
    y = D.grouped_product(codes, scales, None, [0, 1, 2, 4], packed, False, before)
    assert np.array_equal(y[3], D.nvfp4_product(codes, packed[2], False, scales)[3]) and (y[4:] == 9).all()
