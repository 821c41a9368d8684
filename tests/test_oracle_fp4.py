"""Pins of oracle.fp4: code tables, rounding against brute force, block scales, invariants and
planted mistakes. CPU only."""

import numpy as np
import pytest

import oracle as O
from oracle import fp4
from workloads import bf16_bits


def test_e2m1_table_and_rounding():
    # from the bit fields: exponent 0 holds 0 and 0.5, else (1 + m/2) * 2^(e - 1)
    for c in range(8):
        e, m = c >> 1, c & 1
        assert O.E2M1[c] == (0.5 * m if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1))
    # borders go to the even code, values beside them to the nearest
    for lo in range(7):
        mid = (O.E2M1[lo] + O.E2M1[lo + 1]) / 2
        assert O.e2m1_round(mid) == (lo if lo % 2 == 0 else lo + 1)
        assert O.e2m1_round(np.nextafter(mid, 0)) == lo
        assert O.e2m1_round(np.nextafter(mid, 9)) == lo + 1
        assert O.e2m1_round(-mid) == 8 + (lo if lo % 2 == 0 else lo + 1)
    assert O.e2m1_round(1e30) == 7 and O.e2m1_round(-1e30) == 15
    assert O.e2m1_round(0.0) == 0 and O.e2m1_round(-0.0) == 8


def test_e8m0_landmarks():
    assert O.e8m0_value(127) == 1.0 and O.e8m0_value(0) == 2.0 ** -127 and O.e8m0_value(254) == 2.0 ** 127
    assert np.isnan(O.e8m0_value(255))


def test_fp32_quotients_decide_no_code():
    """v / s in fp32 lies on a border of E2M1 only where the exact quotient does: for every
    E4M3 significand and border, the fp32 neighbours of border * s keep their side."""
    for sig in range(8, 16):
        s = np.float32(sig / 8)
        for lo in range(7):
            mid = (O.E2M1[lo] + O.E2M1[lo + 1]) / 2
            at = np.float32(mid * float(s))
            assert float(at) == mid * float(s)  # a border times a scale is an fp32 number
            for v in (np.nextafter(at, np.float32(0)), at, np.nextafter(at, np.float32(100))):
                exact = O.e2m1_round(float(v) / float(s))
                assert O.e2m1_round(float(np.float32(v / s))) == exact
                assert np.sign(float(np.float32(v / s)) - mid) == np.sign(float(v) - float(at))


@pytest.mark.parametrize("fmt", [O.FP4_NV, O.FP4_MX])
def test_exact_grid_is_kept(fmt):
    """Values that the format can hold come back as they are."""
    rng = np.random.default_rng(3)
    block = O.fp4_block(fmt)
    rows, nb = 9, 6
    c = rng.integers(0, 16, size=(rows, nb * block), dtype=np.uint8)
    c[:, ::block] = 7  # each block reaches 6
    if fmt == O.FP4_NV:
        # scales whose largest is 448 fix the row scale at 1
        s = rng.integers(0x20, 0x78, size=(rows, nb), dtype=np.uint8)
        s[:, 0] = 0x7E
    else:
        s = rng.integers(1, 254, size=(rows, nb), dtype=np.uint8)
    codes = c[:, 0::2] | (c[:, 1::2] << 4)
    x = O.dequantize_fp4(codes, s, None, fmt)
    if fmt == O.FP4_MX:
        keep = np.isfinite(x.astype(np.float32))
        assert keep.all()
    q, sc, row = O.quantize_fp4(x.astype(np.float32), "f32", fmt)
    assert np.array_equal(sc, s) and np.all(row == 1)
    got = O.dequantize_fp4(q, sc, row, fmt)
    assert np.array_equal(got, x)


def test_row_scale_is_the_least_power_of_two():
    for top in (1.0, 2688.0, np.nextafter(2688.0, 1e9), 1e-30, 3e38, 2688.0 * 2.0 ** -126):
        x = np.zeros((1, 32), dtype=np.float32)
        x[0, 5] = -np.float32(top)
        _, _, row = O.quantize_fp4(x, "f32", O.FP4_NV)
        t, r = float(abs(x[0, 5])), float(row[0])
        assert t <= 2688 * r and (r == 2.0 ** -126 or t > 2688 * r / 2)


def test_error_bounds_and_special_blocks():
    rng = np.random.default_rng(4)
    x = rng.normal(0, 1, size=(6, 256)).astype(np.float32)
    x[1] = 0
    x[2, 3] = np.inf
    x[3, 40] = np.nan
    x[4, 64:96] = 1e-42
    for fmt in (O.FP4_NV, O.FP4_MX):
        q, s, row = O.quantize_fp4(x, "f32", fmt)
        hat = O.dequantize_fp4(q, s, row, fmt)
        b = O.fp4_block(fmt)
        bad = (~np.isfinite(x)).reshape(6, -1, b).any(2).repeat(b, 1)
        assert np.isnan(hat[bad]).all() and np.isfinite(hat[~bad]).all()
        top = np.where(bad, 0, np.abs(x)).reshape(6, -1, b).max(2).repeat(b, 1)
        # half a step at the top is a sixth of 6; MX saturates 8 to 6, a quarter of it
        worst = (1 / 6 + 1 / 16) if fmt == O.FP4_NV else 0.25
        err = np.abs(np.where(bad, 0, hat - x))
        assert np.all(err <= worst * top + 2.0 ** -10 * row[:, None] * (fmt == O.FP4_NV) + 2.0 ** -128)
        assert np.all(hat[1] == 0)
        bf = bf16_bits(np.where(np.isfinite(x), x, 0))
        q2, s2, r2 = O.quantize_fp4(bf, "bf16", fmt)
        assert q2.shape == q.shape and np.isfinite(O.dequantize_fp4(q2, s2, r2, fmt)).all()


def test_tiling_places_every_byte():
    rng = np.random.default_rng(5)
    s = rng.integers(1, 255, size=(300, 7), dtype=np.uint8)
    t = O.tile_scales(s)
    assert t.shape == (3, 2, 512) and (t != 0).sum() == 300 * 7
    back = t.reshape(3, 2, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(384, 8)
    assert np.array_equal(back[:300, :7], s) and not back[300:].any() and not back[:, 7:].any()


MUTANTS = {
    "ties away from zero": ("e2m1_round", lambda v: (np.searchsorted(
        (fp4.E2M1[1:] + fp4.E2M1[:-1]) / 2, np.minimum(np.abs(v), 6.0), side="right") + 8 * np.signbit(v)).astype(np.uint8)),
    "wraps instead of saturating": ("e2m1_round", lambda v, f=fp4.e2m1_round: np.where(np.abs(v) > 7, 0, f(v))),
    "bias 128": ("e8m0_value", lambda c: np.ldexp(1.0, np.asarray(c, dtype=np.int64) - 128)),
    "blocks of 16 for both": ("fp4_block", lambda fmt: 16),
}


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_a_planted_mistake_fails_a_pin(name, monkeypatch):
    attr, fn = MUTANTS[name]
    monkeypatch.setattr(fp4, attr, fn)
    monkeypatch.setattr(O, attr, fn)
    failed = 0
    for pin in (test_e2m1_table_and_rounding, test_e8m0_landmarks, lambda: test_exact_grid_is_kept(O.FP4_MX),
                test_mx_block_is_32):
        try:
            pin()
        except Exception:
            failed += 1
    assert failed


def test_mx_block_is_32():
    x = np.zeros((1, 64), dtype=np.float32)
    x[0, 31], x[0, 32] = 6.0, 0.5
    _, s, _ = O.quantize_fp4(x, "f32", O.FP4_MX)
    assert s.tolist() == [[127, 124]]  # floor(log2 6) - 2 = 0, floor(log2 0.5) - 2 = -3
