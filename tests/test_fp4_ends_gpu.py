"""The 4-bit operators where values leave the middle of their ranges."""

import numpy as np
import pytest

import oracle as O
from helpers import dev, host
from test_fp4_gpu import _check, _packed
from workloads import activations, bf16_bits

pytestmark = pytest.mark.gpu
FMTS = [O.FP4_NV, O.FP4_MX]


@pytest.fixture(scope="module")
def bd():
    from tenant_serving_b200 import build
    build.build()
    import tenant_serving_b200 as m
    return m


def _dtype(out):
    import torch
    return torch.float32 if out == "f32" else torch.bfloat16


def _bound(y, w_hat, x, e, out):
    """Allowed error of y = x w_hat^T whose activations are off by e: fp32 sums over K = 64 steps,
    their joins and the scales (see test_fp4_gpu), and a bf16 result's own rounding."""
    lim = (w_hat.shape[1] / 64 + 16) * 2.0 ** -23 * (np.abs(x) @ np.abs(w_hat).T) + e @ np.abs(w_hat).T
    return lim + (2.0 ** -8 * (np.abs(y) + lim) if out == "bf16" else 0)


def _no_weight_at(wh, cols):
    """The matrix with code 0 or 8 in some columns: (codes, scales, row)."""
    codes = wh[0].copy()
    for c in cols:
        codes[:, c // 2] &= 0x8F if c % 2 else 0xF8
    return codes, wh[1], wh[2]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("t", [5, 70])
def test_linear_keeps_what_stands_beside_a_massive_value(bd, fmt, out, t):
    """One value 4 10^4 times the others, alone in its block and at weights of zero: the result
    is made of the small values of the token's other blocks, which keep their own precision. L limbs
    leave an element at most 2^-(3 L - 2) of its block's largest, and in BD_FP4_NV no less than
    2^-27 (4 limbs) or 2^-33 (6) of the token's largest."""
    rng = np.random.default_rng(t)
    d_out, d_in, at = 130, 1056, 96
    _, wh = _packed(bd, rng, d_out, d_in, fmt)
    wh = _no_weight_at(wh, [at])
    w_hat = O.dequantize_fp4(*wh, fmt)
    assert (w_hat[:, at] == 0).all()
    x = O.decode(activations(rng, t, d_in), "bf16")
    x[:, at: at + O.fp4_block(fmt)] = 0
    x[:, at] = 4e4 * np.abs(x).mean() * rng.uniform(0.5, 1, size=t)
    xb = bf16_bits(x)
    x = O.decode(xb, "bf16")
    b = O.fp4_block(fmt)
    e = np.abs(x).reshape(t, -1, b).max(2).repeat(b, 1) * (2.0 ** -16 if out == "f32" else 2.0 ** -10)
    if fmt == O.FP4_NV:
        e = e + np.abs(x).max(1, keepdims=True) * (2.0 ** -33 if out == "f32" else 2.0 ** -27)
    x[:, at] = e[:, at] = 0   # (what has no weight takes part in nothing)
    y, ws = bd.bd_linear_fp4(dev(wh[0]), dev(O.tile_scales(wh[1])), None if wh[2] is None else dev(wh[2]), dev(xb), fmt,
                             y_dtype=_dtype(out))
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    ref = x @ w_hat.T
    _check(y, ref, _bound(ref, w_hat, x, e, out))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("t", [5, 70])
def test_linear_keeps_what_stands_beside_an_outlier_of_its_block(bd, fmt, out, t):
    """A power of two, 2^13 times the rest, in every block: one limb holds it exactly, and the
    block's others, n the largest of them, have the remaining L - 1: n 2^-(3 (L - 1) - 2)."""
    rng = np.random.default_rng(t)
    d_out, d_in = 130, 1056
    b = O.fp4_block(fmt)
    at = np.arange(0, d_in, b) + rng.integers(0, b, size=d_in // b)
    _, wh = _packed(bd, rng, d_out, d_in, fmt)
    wh = _no_weight_at(wh, at)
    w_hat = O.dequantize_fp4(*wh, fmt)
    x = rng.uniform(0.25, 1, size=(t, d_in)) * rng.choice([-1, 1], size=(t, d_in))
    x[:, at] = 2.0 ** 13
    xb = bf16_bits(x)
    x = O.decode(xb, "bf16")
    x[:, at] = 0
    e = np.abs(x).reshape(t, -1, b).max(2).repeat(b, 1) * (2.0 ** -13 if out == "f32" else 2.0 ** -7)
    if fmt == O.FP4_NV:
        e += 2.0 ** 13 * (2.0 ** -33 if out == "f32" else 2.0 ** -27)
    y, _ = bd.bd_linear_fp4(dev(wh[0]), dev(O.tile_scales(wh[1])), None if wh[2] is None else dev(wh[2]), dev(xb), fmt,
                            y_dtype=_dtype(out))
    ref = x @ w_hat.T
    _check(y, ref, _bound(ref, w_hat, x, e, out))


# rows kernel alone and with K split over a cluster, pair kernel alone and with K split
ENDS = [(130, 256, 7), (64, 4096, 20), (300, 512, 300), (256, 2304, 300)]


def _scaled(rng, n, exponent):
    return (rng.uniform(1, 2, size=n) * 2.0 ** exponent * rng.choice([-1, 1], size=n)).astype(np.float32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("ew,ex", [(115, -110), (-110, 115), (60, 30), (-50, -30)])
@pytest.mark.parametrize("d_out,d_in,t", ENDS)
def test_row_scales_of_opposite_ends(bd, fmt, out, ew, ex, d_out, d_in, t):
    """Huge weights meet tiny tokens and the reverse: no product on the way to a result of
    ordinary size leaves fp32's range."""
    rng = np.random.default_rng(d_in + t)
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    x, xh = _packed(bd, rng, t, d_in, fmt)
    wr, xr = _scaled(rng, d_out, ew), _scaled(rng, t, ex)
    y, ws = bd.bd_matmul_fp4(w[0], w[1], dev(wr), x[0], x[1], dev(xr), fmt, y_dtype=_dtype(out))
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    w_hat, x_hat = O.dequantize_fp4(wh[0], wh[1], wr, fmt), O.dequantize_fp4(xh[0], xh[1], xr, fmt)
    ref = x_hat @ w_hat.T
    assert np.abs(ref).max() < 2.0 ** 127
    _check(y, ref, _bound(ref, w_hat, x_hat, 0 * x_hat, out))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("ew,ex", [(-30, 60), (60, -30)])
@pytest.mark.parametrize("d_out,d_in,t", ENDS)
def test_row_scales_of_tiny_blocks(bd, out, ew, ex, d_out, d_in, t):
    """Block scales of 2^-60 on both sides: sums near 2^-115 that one of the scales would take
    into the subnormals before the other brings them back."""
    rng = np.random.default_rng(d_in + t)
    fmt = O.FP4_MX
    c = [rng.integers(0, 256, size=(n, d_in // 2), dtype=np.uint8) for n in (d_out, t)]
    s = [rng.integers(64, 70, size=(n, d_in // 32), dtype=np.uint8) for n in (d_out, t)]
    wr, xr = _scaled(rng, d_out, ew), _scaled(rng, t, ex)
    y, _ = bd.bd_matmul_fp4(dev(c[0]), dev(O.tile_scales(s[0])), dev(wr), dev(c[1]), dev(O.tile_scales(s[1])), dev(xr), fmt,
                            y_dtype=_dtype(out))
    w_hat, x_hat = O.dequantize_fp4(c[0], s[0], wr, fmt), O.dequantize_fp4(c[1], s[1], xr, fmt)
    ref = x_hat @ w_hat.T
    _check(y, ref, _bound(ref, w_hat, x_hat, 0 * x_hat, out))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d_out,d_in,t", ENDS)
def test_row_scales_of_zero(bd, fmt, d_out, d_in, t):
    """A row or a token whose scale is zero gives zeros, whatever the other's scale."""
    import torch
    rng = np.random.default_rng(t)
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    x, xh = _packed(bd, rng, t, d_in, fmt)
    for ew, ex in ((0, 122), (122, 0)):
        wr, xr = _scaled(rng, d_out, ew), _scaled(rng, t, ex)
        zero = wr if ex else xr
        zero[::3] = 0
        y, _ = bd.bd_matmul_fp4(w[0], w[1], dev(wr), x[0], x[1], dev(xr), fmt, y_dtype=torch.float32)
        y = host(y) if ex else host(y).T
        assert (y[:, ::3] == 0).all()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("ew,ex", [(-140, 12), (12, -140), (-100, -45)])
@pytest.mark.parametrize("d_out,d_in,t", ENDS)
def test_row_scales_of_huge_blocks(bd, out, ew, ex, d_out, d_in, t):
    """Sums near 2^120 that the larger scale would take past fp32's largest number before the
    other, a subnormal, brings them back; two scales whose product is smaller than any number."""
    rng = np.random.default_rng(d_in + t)
    fmt = O.FP4_MX
    c = [rng.integers(0, 256, size=(n, d_in // 2), dtype=np.uint8) for n in (d_out, t)]
    s = [rng.integers(181, 184, size=(n, d_in // 32), dtype=np.uint8) for n in (d_out, t)]
    wr, xr = (2.0 ** ew * np.ones(d_out)).astype(np.float32), (2.0 ** ex * np.ones(t)).astype(np.float32)
    y, _ = bd.bd_matmul_fp4(dev(c[0]), dev(O.tile_scales(s[0])), dev(wr), dev(c[1]), dev(O.tile_scales(s[1])), dev(xr), fmt,
                            y_dtype=_dtype(out))
    w_hat, x_hat = O.dequantize_fp4(c[0], s[0], wr, fmt), O.dequantize_fp4(c[1], s[1], xr, fmt)
    ref = x_hat @ w_hat.T
    _check(y, ref, _bound(ref, w_hat, x_hat, 0 * x_hat, out))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("t", [4, 5, 70])
def test_linear_of_huge_weights_and_tiny_tokens(bd, out, t):
    """Weights of 1e35 as bd_quantize_fp4 holds them, tokens of 1e-30: finite, whether the
    tokens are few enough for the fp32 kernel or go through limbs."""
    rng = np.random.default_rng(t)
    w = (rng.normal(size=(100, 1056)) * 1e35).astype(np.float32)
    q = O.quantize_fp4(w, "f32", O.FP4_NV)
    codes, scales, row, _ = bd.bd_quantize_fp4(dev(w), O.FP4_NV)
    xb = bf16_bits(O.decode(activations(rng, t, 1056), "bf16") * 1e-30)
    x = O.decode(xb, "bf16")
    y, _ = bd.bd_linear_fp4(codes, scales, row, dev(xb), O.FP4_NV, y_dtype=_dtype(out))
    w_hat = O.dequantize_fp4(*q, O.FP4_NV)
    ref = x @ w_hat.T
    e = np.abs(x).reshape(t, -1, 16).max(2).repeat(16, 1) * (2.0 ** -16 if out == "f32" else 2.0 ** -10)
    e = e + np.abs(x).max(1, keepdims=True) * (2.0 ** -33 if out == "f32" else 2.0 ** -27)
    _check(y, ref, _bound(ref, w_hat, x, e, out))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hat", [None, "f32", "bf16"])
def test_blocks_whose_scale_is_zero(bd, fmt, dtype, hat):
    """Negative values, and zeros with a sign, in blocks far below the row's largest: where the
    block scale rounds to zero the codes are 0."""
    x = np.zeros((4, 96), dtype=np.float32)
    x[0, 0], x[0, 16:32], x[0, 48:64] = 1000, -1e-6, -1e-7
    x[1, 5], x[1, 32:48], x[1, 64:] = -2000, -0.0, -1e-6
    x[2] = -0.0
    x[3, :48], x[3, 48:] = 3, np.where(np.arange(48) % 2, -1e-7, 1e-7)
    if dtype == "bf16":
        x = bf16_bits(x)
    elif dtype == "f16":
        x = x.astype(np.float16)
    codes, scales, row, h = bd.bd_quantize_fp4(dev(x, dtype), fmt, hat_dtype=None if hat is None else _dtype(hat))
    c, s, r = O.quantize_fp4(x, dtype, fmt)
    assert np.array_equal(host(scales), O.tile_scales(s)) and np.array_equal(host(codes), c)
    if hat is not None:
        got = host(h)
        got = O.decode(got, "bf16") if hat == "bf16" else got.astype(np.float64)
        ref = O.dequantize_fp4(c, s, r, fmt)
        assert np.array_equal(got, ref) and np.array_equal(np.signbit(got), np.signbit(ref))
