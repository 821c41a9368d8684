"""The persistent 4-bit kernels with several items per CTA, the early loads of the products
behind a rewritten W, calls that allocate nothing, and the largest sizes."""

import numpy as np
import pytest

import oracle as O
from helpers import dev
from test_fp4_gpu import _check, _delta_limit, _limit, _packed, _table
from workloads import activations, bf16_bits, random_tenant

pytestmark = pytest.mark.gpu
FMTS = [O.FP4_NV, O.FP4_MX]


@pytest.fixture(scope="module")
def bd():
    from tenant_serving_b200 import build
    build.build()
    import tenant_serving_b200 as m
    return m


# (mode, group size): chunked and whole-row kinds in turn, so that a CTA meets both
KINDS = [(0, 128), (1, 0), (4, 128), (2, 0), (0, 256), (3, 0), (1, 0), (0, 128), (4, 256)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d_out,d_in,tenants", [(2000, 768, 64), (2310, 256, 70), (1000, 2304, 130)])
def test_deltas_with_many_items_per_cta(bd, fmt, out, d_out, d_in, tenants):
    """At least three items of the delta kernel per CTA, of alternating kinds: rings, banks, scale
    slots and item buffers pass from one item to the next."""
    import torch
    rng = np.random.default_rng(d_in)
    ten = [random_tenant(rng, d_out, d_in, *KINDS[u % len(KINDS)]) for u in range(tenants)]
    for t in ten:
        t["scales"] = (t["scales"].astype(np.float32) * 40).astype(np.float16)
    counts = rng.integers(1, 4, size=tenants)
    counts[::11] = 13
    ids = np.concatenate([np.full(c, u) for u, c in enumerate(counts)] + [np.full(9, -1)]).astype(np.int32)
    per = 5 if out == "f32" else 8
    items = sum(-(-int(c) // per) for c in counts) * -(-d_out // 256)
    assert items >= 3 * 148
    rng.shuffle(ids)
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    xb = activations(rng, len(ids), d_in)
    x = O.decode(xb, "bf16")
    y, ws = bd.bd_apply_multi_fp4(*w, _table(bd, ten), dev(ids), dev(xb), fmt,
                                  y_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    w_hat = O.dequantize_fp4(*wh, fmt)
    yb, lb = _limit(w_hat, x, fmt, "f32", True)
    if out == "bf16":  # four limbs
        b = O.fp4_block(fmt)
        lb = lb + (np.abs(x).reshape(len(x), -1, b).max(2).repeat(b, 1) * 2.0 ** -10) @ np.abs(w_hat).T
    yd, ld = _delta_limit(ten, ids, x, out)
    ref, lim = yb + yd, lb + ld + 2.0 ** -23 * (np.abs(yb) + np.abs(yd))
    _check(y, ref, lim + (2.0 ** -8 * (np.abs(ref) + lim) if out == "bf16" else 0))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("d_out,d_in,t", [(4096, 320, 3000), (4101, 96, 3001)])
def test_matmul_with_several_tiles_per_pair(bd, fmt, out, d_out, d_in, t):
    """More than two 256 x 256 tiles for each pair of CTAs, both accumulators in turn; rows of y on
    whole 16 bytes (bulk stores) and on odd addresses."""
    import torch
    assert -(-d_out // 256) * -(-t // 256) > 148
    rng = np.random.default_rng(d_in)
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    x, xh = _packed(bd, rng, t, d_in, fmt, std=1.0)
    y, ws = bd.bd_matmul_fp4(*w, *x, fmt, y_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    _check(y, *_limit(O.dequantize_fp4(*wh, fmt), O.dequantize_fp4(*xh, fmt), fmt, out, False))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t", [5, 70])
def test_weights_rewritten_before_each_product(bd, fmt, t):
    """Quantise, linear and apply right behind one another on one stream, with enough tokens for
    the tensor-core products, whose first weights are loaded before the kernel in front of them
    is over: every call sees the weights that were written before it."""
    import torch
    rng = np.random.default_rng(41)
    d_out, d_in = 1024, 2048
    xb = dev(activations(rng, t, d_in))
    ws_ = [dev(bf16_bits(rng.normal(0, 0.02, size=(d_out, d_in)))) for _ in range(3)]
    bufs = bd.fp4_buffers(d_out, d_in, fmt, "cuda")
    table = _table(bd, [random_tenant(rng, d_out, d_in, 1)])
    ids = dev(rng.integers(-1, 1, size=t).astype(np.int32))
    work = bd.fp4_workspace(bd.bd_linear_fp4_workspace_size(d_out, d_in, t), "cuda")
    work_a = bd.fp4_workspace(bd.bd_apply_fp4_workspace_size(d_out, d_in, t, 1), "cuda")

    def one(w):
        bd.bd_quantize_fp4(w, fmt, *bufs)
        y, _ = bd.bd_linear_fp4(*bufs, xb, fmt, workspace=work)
        bd.bd_quantize_fp4(w, fmt, *bufs)
        z, _ = bd.bd_apply_multi_fp4(*bufs, table, ids, xb, fmt, workspace=work_a)
        return y, z

    want = []
    for w in ws_:
        r = one(w)
        torch.cuda.synchronize()
        want.append([v.clone() for v in r])
    assert not torch.equal(want[0][0], want[1][0])
    got = [one(ws_[i % 3]) for i in range(30)]
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 3]))


@pytest.mark.parametrize("fmt", FMTS)
def test_calls_with_all_buffers_given_allocate_nothing(bd, fmt):
    import torch
    rng = np.random.default_rng(6)
    w, _ = _packed(bd, rng, 300, 1056, fmt)
    x = dev(activations(rng, 24, 1056))
    table, ids = _table(bd, [random_tenant(rng, 300, 1056, 1)]), dev(np.zeros(24, dtype=np.int32))
    q, hat = bd.fp4_buffers(24, 1056, fmt, "cuda"), torch.empty_like(x)
    y, out = torch.empty((24, 300), device="cuda"), torch.empty((300, 1056), device="cuda")
    ws = bd.fp4_workspace(max(bd.bd_linear_fp4_workspace_size(300, 1056, 24),
                              bd.bd_apply_fp4_workspace_size(300, 1056, 24, 1)), "cuda")
    s = torch.zeros((300, 1056 // O.fp4_block(fmt)), dtype=torch.uint8, device="cuda")
    tiled = torch.empty_like(w[1])

    def run():
        bd.bd_prepare_fp4_scales(s, fmt, 300, 1056, out=tiled)
        bd.bd_quantize_fp4(x, fmt, *q, hat=hat)
        bd.bd_dequantize_fp4(*w, fmt, out=out)
        bd.bd_matmul_fp4(*w, *q, fmt, y=y, workspace=ws)
        bd.bd_linear_fp4(*w, x, fmt, y=y, workspace=ws)
        bd.bd_apply_multi_fp4(*w, table, ids, x, fmt, y=y, workspace=ws)

    run()
    torch.cuda.synchronize()
    n = torch.cuda.memory_stats()["allocation.all.allocated"]
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        run()
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == n
    assert torch.cuda.mem_get_info()[0] == free


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d_out", [70000, 70001])
def test_outputs_past_32_bits(bd, fmt, d_out):
    """The most tokens, 4.6 10^9 outputs: the last rows and tokens of y, and the first."""
    import torch
    rng = np.random.default_rng(9)
    t, d_in = 65536, 32
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    x, xh = _packed(bd, rng, t, d_in, fmt, std=1.0)
    y, ws = bd.bd_matmul_fp4(*w, *x, fmt, y_dtype=torch.bfloat16)
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    w_hat, x_hat = O.dequantize_fp4(*wh, fmt), O.dequantize_fp4(*xh, fmt)
    for ts, rs in ((slice(0, 300), slice(0, 300)), (slice(t - 300, t), slice(d_out - 300, d_out)),
                   (slice(t // 2, t // 2 + 300), slice(d_out // 2, d_out // 2 + 300))):
        _check(y[ts, rs].contiguous(), *_limit(w_hat[rs], x_hat[ts], fmt, "bf16", False))


@pytest.mark.parametrize("fmt", FMTS)
def test_quantise_past_32_bits(bd, fmt):
    """4.3 10^9 values: the last rows as they come out by themselves, and back."""
    import torch
    rows, cols = 1050000, 4128
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for r0 in range(0, rows, 65536):
        n = min(65536, rows - r0)
        x[r0: r0 + n] = torch.randn((n, cols), generator=g, device="cuda", dtype=torch.bfloat16)
    codes, scales, row, hat = bd.bd_quantize_fp4(x, fmt, hat_dtype=torch.bfloat16)
    for r0 in (0, rows // 2, rows - 130):
        r0 = r0 // 128 * 128  # (where a tile of scales starts)
        n = min(192, rows - r0)
        c, s, r, h = bd.bd_quantize_fp4(x[r0: r0 + n], fmt, hat_dtype=torch.bfloat16)
        assert torch.equal(codes[r0: r0 + n], c) and torch.equal(hat[r0: r0 + n], h)
        assert torch.equal(scales[r0 // 128], s[0]) and (row is None or torch.equal(row[r0: r0 + n], r))
    del x
    back = bd.bd_dequantize_fp4(codes, scales, row, fmt)
    assert torch.equal(back[-1000:], hat[-1000:]) and torch.equal(back[:1000], hat[:1000])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_apply_of_the_most_tokens(bd, fmt, out):
    """65536 tokens of 1500 tenants on a small projection."""
    import torch
    rng = np.random.default_rng(12)
    d_out, d_in, t, tenants = 40, 256, 65536, 1500
    ten = [random_tenant(rng, d_out, d_in, *KINDS[u % len(KINDS)]) for u in range(tenants)]
    ids = rng.integers(-1, tenants, size=t).astype(np.int32)
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    xb = activations(rng, t, d_in)
    y, ws = bd.bd_apply_multi_fp4(*w, _table(bd, ten), dev(ids), dev(xb), fmt,
                                  y_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    pick = np.concatenate([np.arange(200), np.arange(t - 200, t), rng.integers(0, t, size=1600)])
    x, ids, w_hat = O.decode(xb[pick], "bf16"), ids[pick], O.dequantize_fp4(*wh, fmt)
    yb, lb = _limit(w_hat, x, fmt, "f32", True)
    if out == "bf16":
        b = O.fp4_block(fmt)
        lb = lb + (np.abs(x).reshape(len(x), -1, b).max(2).repeat(b, 1) * 2.0 ** -10) @ np.abs(w_hat).T
    yd, ld = _delta_limit(ten, ids, x, out)
    ref, lim = yb + yd, lb + ld + 2.0 ** -23 * (np.abs(yb) + np.abs(yd))
    _check(y[torch.from_numpy(pick).cuda()], ref, lim + (2.0 ** -8 * (np.abs(ref) + lim) if out == "bf16" else 0))
