"""Plain CPU oracle of the decoder-block operators around the quantized
linear layer (TEST INFRASTRUCTURE ONLY): residual + RMS norm + per-token
quantization, the layer's product on unquantized bf16 rows, and the product
grouped by expert.

"RN" is IEEE binary32 round-to-nearest-even (numpy float32 arithmetic); sums
and products are fp64.  The quantizers and formats are
``oracle.qlinear_oracle``'s, pinned there.
"""
from __future__ import annotations

import numpy as np

from . import qlinear_oracle as O

F32 = np.float32


def f32_to_bf16(x: np.ndarray) -> np.ndarray:
    """fp32 -> the nearest bf16 (ties to even) as fp32 values; finite inputs."""
    u = np.ascontiguousarray(x, dtype=F32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(F32)


def rms_norm(x_bits, res_bits, gamma_bits, eps: float):
    """(h, y) as fp32 arrays of bf16 values: h = bf16(RN(x + r)),
    rstd = RN(1 / sqrt(sum h^2 / K + eps)) from fp64,
    y = bf16(RN(RN(h rstd) gamma))."""
    h = O.bf16_bits_to_f32(x_bits)
    if res_bits is not None:
        h = f32_to_bf16(h + O.bf16_bits_to_f32(res_bits))
    mean = (h.astype(np.float64) ** 2).sum(axis=1) / h.shape[1]
    rstd = (1.0 / np.sqrt(mean + np.float64(F32(eps)))).astype(F32)
    y = (h * rstd[:, None]).astype(F32) * O.bf16_bits_to_f32(gamma_bits)[None, :]
    return h, f32_to_bf16(y.astype(F32))


def norm_quantize(x_bits, res_bits, gamma_bits, eps: float, hadamard: bool, qmax: int = O.INT8_QMAX):
    """(h, y, int8 codes, fp32 scales)."""
    h, y = rms_norm(x_bits, res_bits, gamma_bits, eps)
    q, s = O.int8_per_token(O.block_hadamard(y) if hadamard else y, qmax)
    return h, y, q, s


def nvfp4_product(a: np.ndarray, wq: dict, hadamard: bool, row_scale=None) -> np.ndarray:
    """fp64 Y = alpha a W^T on oracle.qlinear_oracle's packed NVFP4 weights:
    alpha = g_w (/128 for rotated weights) times the row's scale.  a: integer
    codes (with row_scale), or unquantized rows (rotated here, in fp64, for
    rotated weights)."""
    a = np.asarray(a, dtype=np.float64)
    if row_scale is None and hadamard:
        a = (a.reshape(-1, O.HADAMARD_N) @ O.sylvester_hadamard(O.HADAMARD_N).astype(np.float64)).reshape(a.shape)
    y = a @ O.nvfp4_dequantize(wq["packed"], wq["sb"]).T * np.float64(wq["g"])
    if hadamard:
        y = y / O.HADAMARD_N
    return y if row_scale is None else y * np.asarray(row_scale, dtype=np.float64)[:, None]


def grouped_product(codes, scales, rows, offsets, experts, hadamard: bool, y: np.ndarray) -> np.ndarray:
    """fp64 rows of Y by expert: Y[r] = codes[src] . experts[e] times the
    scales, src = rows[r] (r without rows), for r in [offsets[e],
    offsets[e+1]); a source row that does not exist gives zeros; rows outside
    every segment keep `y`'s values."""
    out = np.array(y, dtype=np.float64)
    for e, wq in enumerate(experts):
        for r in range(offsets[e], offsets[e + 1]):
            src = r if rows is None else int(rows[r])
            if 0 <= src < len(codes):
                out[r] = nvfp4_product(codes[src:src + 1], wq, hadamard, scales[src:src + 1])[0]
            else:
                out[r] = 0.0
    return out
