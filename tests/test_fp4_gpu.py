"""GPU parity of the microscaled 4-bit operators against the fp64 oracle (oracle.fp4).

Quantisation is bit for bit. Products are held to bounds from arithmetic, with A = sum over
the row of |w_hat| |x|:
  * fp32 accumulation: the products of a K = 64 step and their sum fit fp32 well (4-bit values
    times 4-bit scales); every step adds to the accumulator with an error of at most one
    unit in the last place of a value below A, and so do the joins of a K split; two row
    scales round by half a unit each: (K / 64 + 16) * 2^-23 * A;
  * limbs (bf16 activations), m the block's largest |x|: m * 2^-10 per element for a bf16
    result and m * 2^-16 for an fp32 one, plus 2^-17 of the token's largest in BD_FP4_NV;
  * a bf16 result is rounded by at most 2^-8 of itself.
"""

import numpy as np
import pytest

import oracle as O
from helpers import assert_apply_close, dev, host
from workloads import activations, bf16_bits, random_tenant

pytestmark = pytest.mark.gpu
FMTS = [O.FP4_NV, O.FP4_MX]


@pytest.fixture(scope="module")
def bd():
    from tenant_serving_b200 import build
    build.build()
    import tenant_serving_b200 as m
    return m


def _values(rng, rows, cols, dtype):
    """Rows of unequal size with outliers, a zero row, tiny and huge rows, and values on borders."""
    x = rng.normal(0, 0.02, size=(rows, cols)) * np.exp(rng.normal(0, 1, size=(rows, 1)))
    x[:, ::37] *= 20
    if rows > 6:
        x[1] = 0
        x[2] *= 1e-36 if dtype != "f16" else 1e-4
        x[3] *= 1e36 if dtype != "f16" else 1e3
        x[4] = rng.integers(-24, 25, size=cols) / 4.0          # ties of every border
        x[5, :32] = 0
        x[6, 32:] = 0
    with np.errstate(over="ignore"):
        if dtype == "bf16":
            return bf16_bits(x)
        return x.astype(np.float16 if dtype == "f16" else np.float32)


def _packed(bd, rng, rows, cols, fmt, std=0.02):
    """(device codes, scales, row), (host codes, row-major scales, row): random codes and scales
    with any finite scale among them."""
    codes = rng.integers(0, 256, size=(rows, cols // 2), dtype=np.uint8)
    nb = cols // O.fp4_block(fmt)
    if fmt == O.FP4_NV:
        s = rng.integers(0, 0x7F, size=(rows, nb), dtype=np.uint8)
        row = (std * rng.uniform(0.5, 2, size=rows) / 2 ** 4).astype(np.float32)
        d_row = dev(row)
    else:
        s = rng.integers(110, 125, size=(rows, nb), dtype=np.uint8)
        row, d_row = None, None
    return (dev(codes), dev(O.tile_scales(s)), d_row), (codes, s, row)


def _limit(w_hat, x, fmt, out, limbs):
    """Allowed error per output (see the top of the file). w_hat [d_out, K], x [T, K]."""
    k = w_hat.shape[1]
    aw, ax = np.abs(w_hat), np.abs(x)
    lim = (k / 64 + 16) * 2.0 ** -23 * (ax @ aw.T)
    if limbs:
        b = O.fp4_block(fmt)
        top = ax.reshape(len(x), -1, b).max(2).repeat(b, 1)
        e = top * (2.0 ** -16 if out == "f32" else 2.0 ** -10)
        if fmt == O.FP4_NV:
            e = e + 2.0 ** -17 * ax.max(1, keepdims=True)
        lim += e @ aw.T
    y = x @ w_hat.T
    return y, lim + (2.0 ** -8 * (np.abs(y) + lim) if out == "bf16" else 0)


def _check(y, y_ref, lim):
    y = O.decode(host(y), "bf16") if y.element_size() == 2 else host(y).astype(np.float64)
    err = np.abs(y - y_ref)
    bad = ~(err <= lim)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float((err / np.maximum(lim, 1e-300)).max()))


# -------------------------------------------------------------------------- quantisation
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (7, 96, 0), (130, 416, 8), (300, 4096, 16), (33, 14336, 0),
                                           (9, 20000, 64)])
def test_quantize_is_bit_exact(bd, fmt, dtype, rows, cols, pad):
    import torch
    rng = np.random.default_rng(rows + cols + fmt)
    x = _values(rng, rows, cols, dtype)
    wide = np.zeros((rows, cols + pad), dtype=x.dtype)
    wide[:, :cols] = x
    wide[:, cols:] = np.array(np.inf, dtype=np.float32).astype(np.float16) if dtype == "f16" else x[0, 0]
    dx = dev(wide, dtype)[:, :cols]
    for hat_dtype in (None, torch.float32, torch.bfloat16):
        bufs = bd.fp4_buffers(rows, cols, fmt, "cuda")
        for b in bufs:
            if b is not None:
                b.view(torch.uint8).fill_(0xEE)
        codes, scales, row, hat = bd.bd_quantize_fp4(dx, fmt, *bufs, hat_dtype=hat_dtype)
        c_ref, s_ref, r_ref = O.quantize_fp4(x, dtype, fmt)
        assert np.array_equal(host(scales), O.tile_scales(s_ref))
        assert np.array_equal(host(codes), c_ref)
        if fmt == O.FP4_NV:
            assert np.array_equal(host(row), r_ref)
        ref = O.dequantize_fp4(c_ref, s_ref, r_ref, fmt)
        if hat_dtype is not None:
            got = host(hat)
            got = O.decode(got, "bf16") if hat_dtype == torch.bfloat16 else got.astype(np.float64)
            # exact, but for results among the type's subnormals
            tiny = 2.0 ** -133 if hat_dtype == torch.bfloat16 else 2.0 ** -149
            assert np.all(np.abs(got - ref) <= tiny / 2)
            back = host(bd.bd_dequantize_fp4(codes, scales, row, fmt, out_dtype=hat_dtype))
            assert np.array_equal(back, host(hat))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_infinities_and_nans_stay_in_their_block(bd, fmt, dtype):
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1, size=(5, 160)).astype(np.float32)
    x[0, 3], x[1, 70], x[2, :], x[3, 159] = np.inf, -np.inf, np.nan, np.nan
    if dtype == "bf16":
        bits = (x.view(np.uint32) >> 16).astype(np.uint16)
        bits[np.isnan(x)] = 0x7FC0
        x = bits
    codes, scales, row, hat = bd.bd_quantize_fp4(dev(x, dtype), fmt, hat_dtype=__import__("torch").float32)
    c_ref, s_ref, r_ref = O.quantize_fp4(x, dtype, fmt)
    assert np.array_equal(host(scales), O.tile_scales(s_ref)) and np.array_equal(host(codes), c_ref)
    ref = O.dequantize_fp4(c_ref, s_ref, r_ref, fmt)
    assert np.isnan(ref[2]).all() and np.array_equal(np.isnan(host(hat)), np.isnan(ref))
    assert np.array_equal(host(hat)[~np.isnan(ref)], ref[~np.isnan(ref)].astype(np.float32))


@pytest.mark.parametrize("fmt", FMTS)
def test_dequantize_every_code_and_scale(bd, fmt):
    rows, cols = 256, 32 * 16
    codes = np.tile(np.arange(256, dtype=np.uint8), (rows, 1))
    s = np.arange(rows, dtype=np.uint8)[:, None].repeat(cols // O.fp4_block(fmt), 1)
    if fmt == O.FP4_NV:
        s &= 0x7F  # an unsigned format
    row = np.linspace(-3, 3, rows).astype(np.float32)
    import torch
    for r in (None, row):
        out = host(bd.bd_dequantize_fp4(dev(codes), dev(O.tile_scales(s)), None if r is None else dev(r), fmt,
                                        out_dtype=torch.float32))
        ref = O.dequantize_fp4(codes, s, None, fmt)
        with np.errstate(over="ignore"):
            ref = (ref.astype(np.float32) * (np.float32(1) if r is None else r[:, None]))
        assert np.array_equal(np.isnan(out), np.isnan(ref))
        assert np.array_equal(out[~np.isnan(ref)], ref[~np.isnan(ref)])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols", [(1, 32), (130, 416), (1001, 4128)])
def test_prepare_scales(bd, fmt, rows, cols):
    rng = np.random.default_rng(2)
    s = rng.integers(0, 255, size=(rows, cols // O.fp4_block(fmt)), dtype=np.uint8)
    assert np.array_equal(host(bd.bd_prepare_fp4_scales(dev(s), fmt, rows, cols)), O.tile_scales(s))


# ------------------------------------------------------------------------------ products
SHAPES = [(1, 32, 1), (128, 64, 16), (130, 1056, 7), (257, 608, 77), (1000, 4096, 33), (64, 14336, 129),
          (520, 800, 300), (300, 256, 700), (2050, 320, 1030),
          (770, 2112, 300), (130, 2080, 1000),  # (K split between pairs)
          (1001, 512, 600), (33, 96, 300), (259, 2080, 530)]  # (rows of y on odd addresses)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d_out,d_in,t", SHAPES)
def test_matmul(bd, fmt, out, d_out, d_in, t):
    import torch
    rng = np.random.default_rng(d_out + t)
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    x, xh = _packed(bd, rng, t, d_in, fmt, std=1.0)
    y = torch.full((t + 1, d_out), 7.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    _, ws = bd.bd_matmul_fp4(*w, *x, fmt, y=y[:t])
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    _check(y[:t], *_limit(O.dequantize_fp4(*wh, fmt), O.dequantize_fp4(*xh, fmt), fmt, out, False))
    assert bool((y[t] == 7).all())  # nothing behind the last token


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d_out,d_in,t", SHAPES)
def test_linear(bd, fmt, out, d_out, d_in, t):
    import torch
    rng = np.random.default_rng(d_out + t)
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    x = O.decode(activations(rng, t, d_in), "bf16")
    x *= 2.0 ** rng.integers(-30, 30, size=(t, 1))      # tokens of unequal size
    x[:, ::29] *= 64                                     # outliers
    x[t // 2] = 0
    xb = bf16_bits(x)
    x = O.decode(xb, "bf16")
    y = torch.full((t + 1, d_out), 7.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    _, ws = bd.bd_linear_fp4(*w, dev(xb), fmt, y=y[:t])
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    _check(y[:t], *_limit(O.dequantize_fp4(*wh, fmt), x, fmt, out, True))
    assert bool((y[t] == 7).all()) and bool((y[t // 2] == 0).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d_out,d_in", [(1, 32), (33, 4128), (257, 608), (300, 8224)])
def test_few_tokens(bd, fmt, out, d_out, d_in):
    """1 to 4 tokens on small weights: fp32 products, no limbs; 5 tokens for comparison. An
    infinity or a NaN stays with its token, a NaN block with its row."""
    import torch
    rng = np.random.default_rng(d_in)
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    w_hat = O.dequantize_fp4(*wh, fmt)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    xb = activations(rng, 5, d_in)
    x = O.decode(xb, "bf16")
    for t in range(1, 6):
        y, ws = bd.bd_linear_fp4(*w, dev(xb[:t]), fmt, y_dtype=dt)
        _check(y, *_limit(w_hat, x[:t], fmt, out, t > 4))
        assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    xn = xb[:4].copy()
    xn[1, d_in // 2], xn[3, d_in - 1] = 0xFF80, 0x7FC0
    y, _ = bd.bd_linear_fp4(*w, dev(xn), fmt, y_dtype=dt)
    clean, _ = bd.bd_linear_fp4(*w, dev(xb[:4]), fmt, y_dtype=dt)
    assert torch.isnan(y[[1, 3]]).all() and torch.equal(y[[0, 2]], clean[[0, 2]])
    s = wh[1].copy()
    s[d_out // 2, -1] = 0x7F if fmt == O.FP4_NV else 0xFF
    y, _ = bd.bd_linear_fp4(w[0], dev(O.tile_scales(s)), w[2], dev(xb[:4]), fmt, y_dtype=dt)
    keep = [o for o in range(d_out) if o != d_out // 2]
    assert torch.isnan(y[:, d_out // 2]).all() and torch.equal(y[:, keep], clean[:, keep])


@pytest.mark.parametrize("fmt", FMTS)
def test_few_tokens_at_the_ends_of_fp32(bd, fmt):
    """A token whose unscaled sums pass fp32's largest number beside a tiny one and a NaN."""
    import torch
    rng = np.random.default_rng(3)
    w, wh = _packed(bd, rng, 65, 4128, fmt)
    xb = bf16_bits(O.decode(activations(rng, 4, 4128), "bf16") * 2.0 ** np.array([[116], [-100], [0], [0]]))
    xb[2, 9] = 0x7FC0
    y, _ = bd.bd_linear_fp4(*w, dev(xb), fmt, y_dtype=torch.float32)
    keep = [0, 1, 3]
    x = O.decode(xb, "bf16")[keep]
    _check(y[keep], *_limit(O.dequantize_fp4(*wh, fmt), x, fmt, "f32", False))
    assert torch.isnan(y[2]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_wide_rows_and_row_scales_of_a_checkpoint(bd, fmt):
    """One fp32 scale per tensor that is no power of two, in either format, and negative rows."""
    rng = np.random.default_rng(8)
    w, wh = _packed(bd, rng, 200, 512, fmt)
    x, xh = _packed(bd, rng, 50, 512, fmt)
    import torch
    r = np.where(np.arange(200) % 3 == 0, -0.0123, 0.0123).astype(np.float32)
    y, _ = bd.bd_matmul_fp4(w[0], w[1], dev(r), *x, fmt, y_dtype=torch.float32)
    _check(y, *_limit(O.dequantize_fp4(wh[0], wh[1], r, fmt), O.dequantize_fp4(*xh, fmt), fmt, "f32", False))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t", [5, 200])
def test_nans_reach_their_rows_and_tokens_only(bd, fmt, t):
    import torch
    rng = np.random.default_rng(3)
    nan = 0x7F if fmt == O.FP4_NV else 0xFF
    w, wh = _packed(bd, rng, 150, 256, fmt)
    x, xh = _packed(bd, rng, t, 256, fmt)
    ws, xs = wh[1].copy(), xh[1].copy()
    ws[140, 2] = nan
    xs[3, 1] = nan
    y, _ = bd.bd_matmul_fp4(w[0], dev(O.tile_scales(ws)), w[2], x[0], dev(O.tile_scales(xs)), x[2], fmt,
                            y_dtype=torch.float32)
    want = np.zeros((t, 150), dtype=bool)
    want[:, 140] = True
    want[3] = True
    assert np.array_equal(np.isnan(host(y)), want)
    xb = activations(rng, t, 256)
    xb[1, 100], xb[2, 7] = 0x7F80, 0x7FC0  # an infinity, a NaN
    y, _ = bd.bd_linear_fp4(*w, dev(xb), fmt, y_dtype=torch.float32)
    want = np.zeros((t, 150), dtype=bool)
    want[1:3] = True
    assert np.array_equal(np.isnan(host(y)), want)


def test_no_tokens(bd):
    import torch
    rng = np.random.default_rng(3)
    w, _ = _packed(bd, rng, 64, 64, O.FP4_NV)
    n = bd.bd_launch_count()
    y, _ = bd.bd_linear_fp4(*w, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), O.FP4_NV)
    assert y.shape == (0, 64)
    e = torch.empty((0, 32), dtype=torch.uint8, device="cuda")
    y, _ = bd.bd_matmul_fp4(*w, e, e, None, O.FP4_NV)
    assert y.shape == (0, 64) and bd.bd_launch_count() == n


# ---------------------------------------------------------------------- use as it is used
def _table(bd, tenants):
    recs = []
    for t in tenants:
        s, sc = dev(t["signs"]), dev(t["scales"])
        d_out, wpr = t["signs"].shape
        s, sc = bd.bd_prepare_tenant(s, sc, t["mode"], t["group_size"], d_out, wpr * 32)
        recs.append((s, sc, t["mode"], t["group_size"], 1))
    return bd.TenantTable(recs, "cuda")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d_out,d_in,B,counts", [
    (1100, 640, 1, None), (513, 544, 40, None), (700, 512, 300, (20, 3, 1, 0, 12)), (256, 1024, 700, None),
    (130, 4096, 64, (64,))])
def test_apply_matches_oracle(bd, fmt, d_out, d_in, B, counts):
    import torch
    rng = np.random.default_rng(7 * d_out + B)
    w = bf16_bits(rng.normal(0, 0.02, size=(d_out, d_in)))
    T = 5
    G = 128 if d_in % 128 == 0 else 32
    tenants = [random_tenant(rng, d_out, d_in, u % 4, G) for u in range(T)]
    if counts is None:
        ids = rng.integers(-1, T, size=B).astype(np.int32)
    else:
        ids = np.concatenate([np.full(c, u, dtype=np.int32) for u, c in enumerate(counts)])
        ids = np.concatenate([ids, np.full(B - len(ids), -1, dtype=np.int32)])
        rng.shuffle(ids)
    x = activations(rng, B, d_in)
    codes, scales, row, _ = bd.bd_quantize_fp4(dev(w), fmt)
    q = O.quantize_fp4(w, "bf16", fmt)
    y_ref = O.apply_multi_fp4(*q, fmt, tenants, ids, x, "bf16")
    y, ws = bd.bd_apply_multi_fp4(codes, scales, row, _table(bd, tenants), dev(ids), dev(x), fmt)
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    assert_apply_close(O.decode(host(y), "bf16"), y_ref)
    y32, _ = bd.bd_apply_multi_fp4(codes, scales, row, _table(bd, tenants), dev(ids), dev(x), fmt, y_dtype=torch.float32)
    assert_apply_close(host(y32), y_ref, per_token=True)


def _delta_limit(tenants, ids, x, out):
    """Delta_hat x and its allowed error: limbs as for bf16 activations (blocks of 32; COL scales
    are multiplied into the activations first), fp32 sums over chunks of 8 or more columns, and
    two units in the last place for the scales' products."""
    d_out, d_in = tenants[0]["signs"].shape[0], x.shape[1]
    y, lim = np.zeros((len(x), d_out)), np.zeros((len(x), d_out))
    eps = 2.0 ** -16 if out == "f32" else 2.0 ** -10
    deltas = [O.reconstruct(t["signs"], t["scales"].astype(np.float64), t["mode"], t["group_size"], d_out, d_in)
              for t in tenants]
    for t, u in enumerate(ids):
        if u < 0:
            continue
        ten, d = tenants[u], deltas[u]
        ax = np.abs(x[t]) * (np.asarray(ten["scales"], dtype=np.float64) if ten["mode"] == 2 else 1.0)
        ad = np.ones_like(d) if ten["mode"] == 2 else np.abs(d)
        top = ax.reshape(-1, 32).max(1).repeat(32)
        y[t] = d @ x[t]
        lim[t] = ad @ (eps * top + 2.0 ** -126) + ((d_in / 8 + 16) * 2.0 ** -23 + 2.0 ** -22) * (ad @ ax)
    return y, lim


MODES = [(0, 128), (0, 256), (0, 32), (1, 0), (2, 0), (3, 0), (4, 128), (4, 512), (4, 64)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d_out,d_in", [(300, 512), (520, 1536), (129, 2560)])
def test_deltas_of_every_kind(bd, fmt, out, d_out, d_in):
    """Every scale mode, group sizes that the 4-bit product takes and that it leaves to the lookup
    kernel, row-major records beside tiled ones, and 1 to 33 tokens of a tenant in a batch."""
    import torch
    rng = np.random.default_rng(d_out + d_in)
    tenants = [random_tenant(rng, d_out, d_in, m, g or 128) for m, g in MODES] + [random_tenant(rng, d_out, d_in, 0, 128)]
    for t in tenants:  # larger than in use: the delta is what is held to its bound here
        t["scales"] = (t["scales"].astype(np.float32) * 40).astype(np.float16)
    counts = [3, 2, 1, 9, 8, 33, 5, 17, 4, 6]
    ids = np.concatenate([np.full(c, u) for u, c in enumerate(counts)] + [np.full(7, -1)]).astype(np.int32)
    rng.shuffle(ids)
    recs = []
    for u, t in enumerate(tenants):
        sg, sc = dev(t["signs"]), dev(t["scales"])
        if u < len(MODES):
            sg, sc = bd.bd_prepare_tenant(sg, sc, t["mode"], t["group_size"], d_out, d_in)
        recs.append((sg, sc, t["mode"], t["group_size"], bd.BD_LAYOUT_TILED if u < len(MODES) else bd.BD_LAYOUT_ROWMAJOR))
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    x = O.decode(activations(rng, len(ids), d_in), "bf16") * 2.0 ** rng.integers(-20, 20, size=(len(ids), 1))
    x[:, ::31] *= 32
    xb = bf16_bits(x)
    x = O.decode(xb, "bf16")
    y, ws = bd.bd_apply_multi_fp4(*w, bd.TenantTable(recs, "cuda"), dev(ids), dev(xb), fmt,
                                  y_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    yb, lb = _limit(O.dequantize_fp4(*wh, fmt), x, fmt, "f32", True)
    if out == "bf16":  # four limbs
        e = np.abs(x).reshape(len(x), -1, O.fp4_block(fmt)).max(2).repeat(O.fp4_block(fmt), 1) * 2.0 ** -10
        lb = lb + e @ np.abs(O.dequantize_fp4(*wh, fmt)).T
    yd, ld = _delta_limit(tenants, ids, x, out)
    ref, lim = yb + yd, lb + ld + 2.0 ** -23 * (np.abs(yb) + np.abs(yd))
    _check(y, ref, lim + (2.0 ** -8 * (np.abs(ref) + lim) if out == "bf16" else 0))


@pytest.mark.parametrize("fmt", FMTS)
def test_apply_status_and_limits(bd, fmt):
    """An id out of range and a bad record are reported, their tokens get the base; infinities
    and NaN stay with their token; no tenants at all; one token of one tenant."""
    import torch
    rng = np.random.default_rng(31)
    d_out, d_in = 200, 512
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    ten = [random_tenant(rng, d_out, d_in, 0, 128) for _ in range(2)]
    table = _table(bd, ten)
    xb = activations(rng, 6, d_in)
    base, _ = bd.bd_linear_fp4(*w, dev(xb), fmt, y_dtype=torch.float32)
    ids = np.array([0, 7, -1, 1, -5, 0], dtype=np.int32)
    y, ws = bd.bd_apply_multi_fp4(*w, table, dev(ids), dev(xb), fmt, y_dtype=torch.float32)
    assert bd.bd_get_status(ws) == (bd.BD_ERR_TENANT_RANGE, bd.BD_DEV_TENANT_RANGE)
    assert torch.equal(y[[1, 2, 4]], base[[1, 2, 4]]) and not torch.equal(y[0], base[0])
    bad = bd.TenantTable([(dev(ten[0]["signs"]), dev(ten[0]["scales"]), 0, 96, 1)], "cuda")
    y, ws = bd.bd_apply_multi_fp4(*w, bad, dev(np.zeros(6, dtype=np.int32)), dev(xb), fmt, y_dtype=torch.float32)
    assert bd.bd_get_status(ws)[0] == bd.BD_ERR_TENANT_RECORD and torch.equal(y, base)
    y, ws = bd.bd_apply_multi_fp4(*w, bd.TenantTable([], "cuda"), dev(np.full(6, -1, dtype=np.int32)), dev(xb), fmt,
                                  y_dtype=torch.float32)
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0) and torch.equal(y, base)
    xn = xb.copy()
    xn[0, 5], xn[3, 300] = 0x7F80, 0x7FC0
    ids = np.array([0, 0, -1, 1, 1, 0], dtype=np.int32)
    y, _ = bd.bd_apply_multi_fp4(*w, table, dev(ids), dev(xn), fmt, y_dtype=torch.float32)
    clean, _ = bd.bd_apply_multi_fp4(*w, table, dev(ids), dev(xb), fmt, y_dtype=torch.float32)
    assert torch.isnan(y[[0, 3]]).all() and torch.equal(y[[1, 2, 4, 5]], clean[[1, 2, 4, 5]])
    one, _ = bd.bd_apply_multi_fp4(*w, table, dev(ids[:1]), dev(xb[:1]), fmt, y_dtype=torch.float32)
    # One token's base product is made in fp32, six tokens' from limbs: the two differ by what
    # six limbs leave of each value and by the two products' fp32 sums (_limit has both), and the
    # sum with the delta rounds by 2^-24 of itself in each.
    _, lim = _limit(O.dequantize_fp4(*wh, fmt), O.decode(xb[:1], "bf16"), fmt, "f32", True)
    clean = host(clean)[:1].astype(np.float64)
    _check(one, clean, 2 * lim + 2.0 ** -23 * np.abs(clean))


@pytest.mark.parametrize("fmt", FMTS)
def test_back_to_back(bd, fmt):
    """Quantise, product and apply right behind one another on one stream, with new weights each
    time in the same buffers: every product sees the weights that were written before it."""
    import torch
    rng = np.random.default_rng(41)
    d_out, d_in = 1024, 2048
    xb = dev(activations(rng, 3, d_in))
    ws_ = [dev(bf16_bits(rng.normal(0, 0.02, size=(d_out, d_in)))) for _ in range(3)]
    bufs = bd.fp4_buffers(d_out, d_in, fmt, "cuda")
    table = _table(bd, [random_tenant(rng, d_out, d_in, 1)])
    ids = dev(np.array([0, -1, 0], dtype=np.int32))
    work = bd.fp4_workspace(bd.bd_linear_fp4_workspace_size(d_out, d_in, 3), "cuda")
    work_a = bd.fp4_workspace(bd.bd_apply_fp4_workspace_size(d_out, d_in, 3, 1), "cuda")

    def one(w):
        bd.bd_quantize_fp4(w, fmt, *bufs)
        y, _ = bd.bd_linear_fp4(*bufs, xb, fmt, workspace=work)
        z, _ = bd.bd_apply_multi_fp4(*bufs, table, ids, xb, fmt, workspace=work_a)
        return y, z

    want = []
    for w in ws_:
        r = one(w)
        torch.cuda.synchronize()
        want.append([t.clone() for t in r])
    got = [one(ws_[i % 3]) for i in range(30)]
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 3]))


@pytest.mark.parametrize("fmt", FMTS)
def test_compress_against_the_served_base_and_serve(bd, fmt):
    """Quantise a base, take a fine-tune's delta against what is served, serve the tenant
    over the 4-bit base: the whole run against the oracle's."""
    import torch
    rng = np.random.default_rng(21)
    d_out, d_in, B = 384, 512, 11
    base = bf16_bits(rng.normal(0, 0.02, size=(d_out, d_in)))
    fine = bf16_bits(O.decode(base, "bf16") + rng.normal(0, 0.001, size=(d_out, d_in)))
    codes, scales, row, hat = bd.bd_quantize_fp4(dev(base), fmt, hat_dtype=torch.bfloat16)
    assert torch.equal(bd.bd_dequantize_fp4(codes, scales, row, fmt), hat)
    cfg = bd.compress_cfg(mode=bd.BD_SCALE_GROUP, group_size=128)
    signs, sc, _ = bd.bd_compress(hat, dev(fine), cfg)
    sg, sct = bd.bd_prepare_tenant(signs, sc.half(), bd.BD_SCALE_GROUP, 128, d_out, d_in)
    table = bd.TenantTable([(sg, sct, bd.BD_SCALE_GROUP, 128, bd.BD_LAYOUT_TILED)], "cuda")
    ids = np.array([0, -1] * B, dtype=np.int32)[:B]
    x = activations(rng, B, d_in)
    y, ws = bd.bd_apply_multi_fp4(codes, scales, row, table, dev(ids), dev(x), fmt, y_dtype=torch.float32)
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    q = O.quantize_fp4(base, "bf16", fmt)
    hat_ref = O.dequantize_fp4(*q, fmt)
    assert np.array_equal(O.decode(host(hat), "bf16"), hat_ref)
    delta = O.decode(fine, "bf16") - hat_ref
    s_ref = np.abs(delta).reshape(d_out, -1, 128).mean(2)
    tenant = {"signs": host(signs), "scales": s_ref.astype(np.float16), "scale_dtype": "f16", "mode": 0, "group_size": 128}
    assert np.array_equal(host(signs), O.pack_bits(delta >= 0))
    assert_apply_close(host(y), O.apply_multi_fp4(*q, fmt, [tenant], ids, x, "bf16"), per_token=True)
    # tokens of the base alone are those of the linear, and merging agrees
    lin, _ = bd.bd_linear_fp4(codes, scales, row, dev(x), fmt, y_dtype=torch.float32)
    assert_apply_close(host(y)[1::2], host(lin)[1::2].astype(np.float64), tol=1e-6, per_token=True)


@pytest.mark.parametrize("fmt", FMTS)
def test_graphs_and_streams(bd, fmt):
    """Captured and replayed with new inputs, two graphs on one workspace one after the other,
    and two streams at once with a workspace each: the eager results, bit for bit."""
    import torch
    rng = np.random.default_rng(5)
    w, _ = _packed(bd, rng, 1100, 1056, fmt)
    xs = [dev(activations(rng, 24, 1056)) for _ in range(3)]
    table = _table(bd, [random_tenant(rng, 1100, 1056, m, 32) for m in (1, 2, 0)])
    ids = dev(rng.integers(-1, 3, size=24).astype(np.int32))

    def chain(x, bufs):
        bd.bd_quantize_fp4(x, fmt, *bufs["q"])
        bd.bd_matmul_fp4(*w, *bufs["q"], fmt, y=bufs["y4"], workspace=bufs["ws4"])
        bd.bd_linear_fp4(*w, x, fmt, y=bufs["y"], workspace=bufs["ws"])
        bd.bd_apply_multi_fp4(*w, table, ids, x, fmt, y=bufs["ya"], workspace=bufs["wsa"])
        return bufs["y4"], bufs["y"], bufs["ya"]

    def buffers():
        return {"q": bd.fp4_buffers(24, 1056, fmt, "cuda"),
                "y4": torch.empty((24, 1100), dtype=torch.bfloat16, device="cuda"),
                "y": torch.empty((24, 1100), dtype=torch.float32, device="cuda"),
                "ws4": bd.fp4_workspace(bd.bd_matmul_fp4_workspace_size(1100, 1056, 24), "cuda"),
                "ws": bd.fp4_workspace(bd.bd_linear_fp4_workspace_size(1100, 1056, 24), "cuda"),
                "ya": torch.empty((24, 1100), dtype=torch.bfloat16, device="cuda"),
                "wsa": bd.fp4_workspace(bd.bd_apply_fp4_workspace_size(1100, 1056, 24, 3), "cuda")}

    want = [[t.clone() for t in chain(x, buffers())] for x in xs]
    shared = buffers()
    own_x = xs[0].clone()
    graphs = []
    side = torch.cuda.Stream()
    for x in (own_x, xs[1]):
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            chain(x, shared)
        graphs.append(g)
    for i, w_ in ((0, want[0]), (1, want[1]), (0, want[0])):
        graphs[i].replay()
        assert all(torch.equal(a, b) for a, b in zip((shared["y4"], shared["y"], shared["ya"]), w_))
    own_x.copy_(xs[2])
    graphs[0].replay()
    assert all(torch.equal(a, b) for a, b in zip((shared["y4"], shared["y"], shared["ya"]), want[2]))

    streams = [torch.cuda.Stream() for _ in range(2)]
    bufs = [buffers() for _ in streams]
    torch.cuda.synchronize()
    for rep in range(5):
        for s, b, x in zip(streams, bufs, xs):
            with torch.cuda.stream(s):
                chain(x, b)
    torch.cuda.synchronize()
    for b, w_ in zip(bufs, want):
        assert all(torch.equal(p, q) for p, q in zip((b["y4"], b["y"], b["ya"]), w_))


def test_wrapper_refusals(bd):
    import torch
    c, s, r = bd.fp4_buffers(64, 128, O.FP4_NV, "cuda")
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: bd.bd_linear_fp4(c, s, r, x[:, :64], O.FP4_NV),
                 lambda: bd.bd_linear_fp4(c, s, r, torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")[:, ::2], O.FP4_NV),
                 lambda: bd.bd_linear_fp4(c, s[:, :1].contiguous(), r, x, O.FP4_NV),
                 lambda: bd.bd_linear_fp4(c, s, r[:3].contiguous(), x, O.FP4_NV),
                 lambda: bd.bd_linear_fp4(c, s, r, x, O.FP4_NV, y=torch.empty((4, 63), device="cuda")),
                 lambda: bd.bd_quantize_fp4(x.t(), O.FP4_NV),
                 lambda: bd.bd_quantize_fp4(x[:, :72], O.FP4_NV),
                 lambda: bd.bd_matmul_fp4(c, s, r, *bd.fp4_buffers(4, 64, O.FP4_NV, "cuda"), O.FP4_NV),
                 lambda: bd.bd_prepare_fp4_scales(s, O.FP4_NV, 64, 96)):
        with pytest.raises(bd.BitDeltaError):
            call()
    with pytest.raises(TypeError):
        bd.bd_linear_fp4(c, s, r, x.half(), O.FP4_NV)
    with pytest.raises(TypeError):
        bd.bd_linear_fp4(c, s, r.double(), x, O.FP4_NV)
    with pytest.raises(ValueError):
        bd.bd_linear_fp4(c, s.cpu(), r, x, O.FP4_NV)
