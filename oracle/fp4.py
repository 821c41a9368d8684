"""float64 reference of microscaled 4-bit matrices: quantisation, the tiled layout of block
scales, and products of quantised matrices.

TEST INFRASTRUCTURE ONLY, like the rest of this package: the product path never imports
it and it never imports the product.

"BitDelta Guide", "3. Quantized Base Model Compatibility (BitDelta + GPTQ / QuIP#)";
"Per-Axis Weight Deltas for Frequent Model Updates", Future Directions: INT4/FP8 co-design.
The pages name no 4-bit format; the ones taken here are those that the GPU multiplies:

* Elements: OCP E2M1, 1 sign bit, 2 exponent bits with bias 1, 1 mantissa bit: magnitudes
  0, 0.5, 1, 1.5, 2, 3, 4, 6 for codes 0..7. Two per byte, the even column in the low nibble.
* ``FP4_MX`` (OCP Microscaling MXFP4): blocks of 32 columns, scale 2^(byte - 127) (E8M0, 255 is
  NaN). e = floor(log2(max|block|)) - 2, where 2 is the exponent of E2M1's largest value,
  kept in [-127, 127]; codes round x / 2^e to nearest, ties to the even code, saturating.
* ``FP4_NV``: blocks of 16 columns, scale an E4M3 value without its sign, and one fp32 power of
  two per row, the least 2^k with max|row| <= 6 * 448 * 2^k and -126 <= k <= 126 (k = 0 for a
  zero row). scale = E4M3(max|block / 2^k| / 6), codes = E2M1(x / 2^k / scale); both quotients
  are taken in fp32, which decides no code differently from exact quotients (pinned).
* A block with an infinity or a NaN has the NaN scale (0x7F, 0xFF) and codes 0; the other
  blocks are those of the row without it.
* Scale bytes are stored in tiles of 128 rows x 4 blocks: byte (r % 32) * 16 + (r // 32) * 4 + c.
"""

from __future__ import annotations

import numpy as np

from .bitdelta import apply_multi, decode
from .fp8 import e4m3_round, e4m3_value

FP4_NV, FP4_MX = 0, 1
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def fp4_block(fmt: int) -> int:
    return {FP4_NV: 16, FP4_MX: 32}[fmt]


def e2m1_round(v) -> np.ndarray:
    """E2M1 codes of real values: nearest magnitude, ties to the even code, saturation at 6,
    sign kept (also of a zero)."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), 6.0)
    d = np.abs(a[..., None] - E2M1)
    best = d.min(axis=-1, keepdims=True)
    near = d == best
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    return (pick + 8 * np.signbit(v)).astype(np.uint8)


def e8m0_value(code) -> np.ndarray:
    c = np.asarray(code, dtype=np.uint8).astype(np.int64)
    return np.where(c == 255, np.nan, np.ldexp(1.0, c - 127))


def _widen(x, dtype):
    if dtype == "f16":
        return np.asarray(x, dtype=np.float16).astype(np.float64)
    return decode(x, dtype)


def quantize_fp4(x, dtype: str, fmt: int):
    """(codes uint8 [rows, cols/2], scales uint8 [rows, cols/B], row scales float32 [rows])."""
    with np.errstate(invalid="ignore", over="ignore"):
        x = _widen(x, dtype)
    rows, cols = x.shape
    block = fp4_block(fmt)
    b = x.reshape(rows, cols // block, block)
    bad = ~np.isfinite(b).all(axis=2)
    finite = np.where(np.isfinite(x), x, 0.0)
    row = np.ones(rows)
    if fmt == FP4_NV:
        for o, top in enumerate(np.abs(finite).max(axis=1)):
            if top > 0:
                k = -126
                while k < 126 and top > 2688.0 * 2.0 ** k:
                    k += 1
                row[o] = 2.0 ** k
    v = np.where(bad[:, :, None], 0.0, b) / row[:, None, None]
    top = np.abs(v).max(axis=2)
    if fmt == FP4_NV:
        scales = e4m3_round((top.astype(np.float32) / np.float32(6.0)).astype(np.float32))
        s = e4m3_value(scales)
        q = np.where(s[:, :, None] > 0, v / np.where(s > 0, s, 1.0)[:, :, None], 0.0)
        scales = np.where(bad, 0x7F, scales)
    else:
        e = np.full(top.shape, -127, dtype=np.int64)
        nz = top > 0
        e[nz] = np.clip(np.frexp(top[nz])[1] - 1 - 2, -127, 127)
        q = v / np.ldexp(1.0, e)[:, :, None]
        scales = np.where(bad, 0xFF, e + 127)
    c = np.where(bad[:, :, None], 0, e2m1_round(q)).astype(np.uint8).reshape(rows, cols)
    return c[:, 0::2] | (c[:, 1::2] << 4), scales.astype(np.uint8), row.astype(np.float32)


def tile_scales(scales) -> np.ndarray:
    """Row-major scale bytes -> [row tiles, block tiles, 512], padding zero."""
    rows, nb = scales.shape
    out = np.zeros((-(-rows // 128), -(-nb // 4), 512), dtype=np.uint8)
    for r in range(rows):
        for c in range(nb):
            out[r // 128, c // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4] = scales[r, c]
    return out


def dequantize_fp4(codes, scales, row, fmt: int) -> np.ndarray:
    """X_hat in float64 from codes, row-major scale bytes and row scales (or None)."""
    c = np.stack((codes & 15, codes >> 4), axis=2).reshape(codes.shape[0], -1)
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    s = e4m3_value(scales) if fmt == FP4_NV else e8m0_value(scales)
    v = v * np.repeat(s, fp4_block(fmt), axis=1)
    return v if row is None else v * np.asarray(row, dtype=np.float64)[:, None]


def apply_multi_fp4(codes, scales, row, fmt, tenants, tenant_ids, x, x_dtype: str, rows=None):
    """y_t = W_hat x_t + Delta_hat_u x_t with the quantised base (float64)."""
    return apply_multi(dequantize_fp4(codes, scales, row, fmt), "f64", tenants, tenant_ids, x, x_dtype, rows=rows)
