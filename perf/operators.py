"""Timing cases of the microscaled 4-bit operators: quantise, dequantise, the two products and
the multi-tenant apply over a 4-bit base.

A matrix is held as E2M1 codes (two per byte, the even column in the low nibble), one scale
per block of 16 (UE4M3, format "nv") or 32 (E8M0, format "mx") columns and, in "nv", one fp32
scale per row. Block scales sit in tiles of 128 rows x 4 scales (512 bytes): row r, scale c of
a tile at byte (r % 32) * 16 + (r / 32) * 4 + c.
"""

import math

import numpy as np
import torch

own = False

BLOCK = {"nv": 16, "mx": 32}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def _bd():
    import tenant_serving_b200 as bd
    return bd


def _fmt(case):
    bd = _bd()
    return bd.BD_FP4_NV if case["fmt"] == "nv" else bd.BD_FP4_MX


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # the widest weight of a layer, quantised once for serving; the quantised values come
        # back too, since the tenants' deltas are taken against them
        {"name": "quantize gate_up nv", "op": "quantize", "fmt": "nv", "rows": 28672, "cols": 4096, "ld": 4096,
         "dtype": "bf16", "hat": "bf16"},
        # a batch's fp32 activations before a 4-bit product, a column range of a wider buffer
        {"name": "quantize tokens mx", "op": "quantize", "fmt": "mx", "rows": 512, "cols": 14336, "ld": 28672,
         "dtype": "f32", "hat": "f32"},
        # a served 4-bit base read back as the bf16 base of a compress run
        {"name": "dequantize up nv", "op": "dequantize", "fmt": "nv", "rows": 14336, "cols": 4096, "out": "bf16"},
        # a ragged matrix back to fp32
        {"name": "dequantize ragged mx", "op": "dequantize", "fmt": "mx", "rows": 1001, "cols": 4128, "out": "f32"},
        # prompts of several requests, activations quantised: the largest product
        {"name": "matmul prompts gate_up nv", "op": "matmul", "fmt": "nv", "rows": 28672, "cols": 4096,
         "tokens": 8192, "out": "bf16"},
        # the serving batch on the long rows of the down projection
        {"name": "matmul batch down mx", "op": "matmul", "fmt": "mx", "rows": 4096, "cols": 14336, "tokens": 512,
         "out": "bf16"},
        # an odd number of tokens on a narrow projection, fp32 result
        {"name": "matmul odd k nv", "op": "matmul", "fmt": "nv", "rows": 1024, "cols": 4096, "tokens": 77,
         "out": "f32"},
        # a single token: latency
        {"name": "linear one token o nv", "op": "linear", "fmt": "nv", "rows": 4096, "cols": 4096, "tokens": 1,
         "out": "bf16"},
        # a small decode batch, fp32 result
        {"name": "linear 20 tokens down mx", "op": "linear", "fmt": "mx", "rows": 4096, "cols": 14336, "tokens": 20,
         "out": "f32"},
        # the serving batch with bf16 activations on the widest projection
        {"name": "linear batch gate_up nv", "op": "linear", "fmt": "nv", "rows": 28672, "cols": 4096, "tokens": 512,
         "out": "bf16"},
        # the decode workload: every token another tenant
        {"name": "apply decode up nv", "op": "apply", "fmt": "nv", "rows": 14336, "cols": 4096, "tokens": 64,
         "tenants": 64, "ids": "each", "scales": "group", "out": "bf16"},
        # the mixed workload: tenants of unequal popularity, some tokens of the base alone
        {"name": "apply mixed qkv mx", "op": "apply", "fmt": "mx", "rows": 6144, "cols": 4096, "tokens": 256,
         "tenants": 32, "ids": "zipf", "scales": "row", "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["quantize", "dequantize", "matmul", "linear", "apply"])
    case = {"op": op, "fmt": rng.choice(["nv", "mx"])}
    cols = 32 * _log_int(rng, 4, 448)
    if op == "quantize":
        case |= {"rows": _log_int(rng, 1, 28672), "cols": cols, "ld": cols + rng.choice([0, 8 * rng.randint(1, 600)]),
                 "dtype": rng.choice(["bf16", "f16", "f32"]), "hat": rng.choice(["bf16", "f32"])}
    elif op == "dequantize":
        case |= {"rows": _log_int(rng, 1, 28672), "cols": cols, "out": rng.choice(["bf16", "f32"])}
    elif op == "apply":
        case |= {"rows": _log_int(rng, 64, 14336), "cols": cols, "tokens": _log_int(rng, 1, 512),
                 "tenants": _log_int(rng, 1, 64), "ids": "zipf", "scales": rng.choice(["group", "row"]),
                 "out": rng.choice(["bf16", "bf16", "f32"])}
        if case["scales"] == "group":
            case["cols"] = 128 * max(1, cols // 128)
    else:
        case |= {"rows": _log_int(rng, 64, 28672), "cols": cols,
                 "tokens": _log_int(rng, 1, 8192 if op == "matmul" else 512), "out": rng.choice(["bf16", "f32"])}
    return case


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for k in w:
            most[k] = max(most.get(k, 0), w[k])
    for _ in range(100):
        case = _draw(rng)
        w = work(case)
        if all(w[k] <= most[k] for k in w):
            return case
    return case


def _zipf(n_tenants):
    p = np.arange(1, n_tenants + 1, dtype=np.float64) ** -1.1
    return p / p.sum()


def _present(case):
    """Tenants that a batch is expected to hold."""
    if case["ids"] == "each":
        return min(case["tokens"], case["tenants"])
    return float((1 - (1 - 0.9 * _zipf(case["tenants"])) ** case["tokens"]).sum())


def work(case):
    n = case["rows"] * case["cols"]
    row_scales = 4 * case["rows"] if case["fmt"] == "nv" else 0
    packed = n / 2 + n / BLOCK[case["fmt"]] + row_scales
    if case["op"] == "quantize":
        return {"bytes": n * (SIZE[case["dtype"]] + SIZE[case["hat"]]) + packed, "flops": 3 * n}
    if case["op"] == "dequantize":
        return {"bytes": n * SIZE[case["out"]] + packed, "flops": 2 * n}
    t = case["tokens"]
    y = t * case["rows"] * SIZE[case["out"]]
    k = t * case["cols"]
    if case["op"] == "matmul":
        x = k / 2 + k / BLOCK[case["fmt"]] + (4 * t if case["fmt"] == "nv" else 0)
        return {"bytes": packed + x + y, "flops": 2 * n * t}
    if case["op"] == "linear":
        return {"bytes": packed + 2 * k + y, "flops": 2 * n * t}
    signs = n / 8 + (n / 128 * 2 if case["scales"] == "group" else 2 * case["rows"])
    return {"bytes": packed + 2 * k + y + 4 * t + _present(case) * signs, "flops": 4 * n * t}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _matrix(rng, rows, cols, std, dtype):
    """Rows of unequal size with a few large columns, as weights and activations have."""
    x = torch.randn((rows, cols), generator=rng, device="cuda") * std
    x *= torch.exp(0.3 * torch.randn((rows, 1), generator=rng, device="cuda"))
    x[:, :: max(1, cols // 8)] *= 10.0
    return x.to(dtype)


def _packed(rng, rows, cols, std, fmt):
    """A quantised matrix as a program holds it: codes, tiled block scales, row scales."""
    codes, scales, row = [], [], []
    for r0 in range(0, rows, 4096):  # (a multiple of the scale tile's 128 rows)
        x = _matrix(rng, min(4096, rows - r0), cols, std, torch.bfloat16)
        q, s, r = _quantise(x, fmt)
        codes.append(_pack(q))
        scales.append(_tile(s, fmt))
        row.append(r)
    return {"codes": torch.cat(codes), "scales": torch.cat(scales),
            "row": torch.cat(row) if fmt == "nv" else None, "rows": rows, "cols": cols}


def prepare(case, seed):
    rng = torch.Generator(device="cuda")
    rng.manual_seed(seed)
    st = {"case": case, "keep": {}}
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "quantize":
        wide = _matrix(rng, rows, case["ld"], 0.02, DTYPE[case["dtype"]])
        st["x"] = wide[:, :cols]
        return st
    st["w"] = _packed(rng, rows, cols, 0.02, case["fmt"])
    if case["op"] == "dequantize":
        return st
    t = case["tokens"]
    if case["op"] == "matmul":
        st["x"] = _packed(rng, t, cols, 1.0, case["fmt"])
        return st
    st["x"] = _matrix(rng, t, cols, 1.0, torch.bfloat16)
    if case["op"] == "apply":
        n = case["tenants"]
        host = np.random.default_rng(seed)
        if case["ids"] == "each":
            ids = host.permutation(max(t, n))[:t] % n
        else:
            ids = host.choice(n, size=t, p=_zipf(n))
            ids[host.random(t) < 0.1] = -1  # the base alone
        st["ids"] = torch.from_numpy(ids.astype(np.int32)).cuda()
        st["signs"] = [torch.randint(-(2 ** 31), 2 ** 31 - 1, (rows, cols // 32), generator=rng, device="cuda",
                                     dtype=torch.int32) for _ in range(n)]
        shape = (rows, cols // 128) if case["scales"] == "group" else (rows,)
        st["scales"] = [(0.0008 * torch.exp(0.1 * torch.randn(shape, generator=rng, device="cuda"))).half()
                        for _ in range(n)]
        st["tokens_of"] = [(u, torch.from_numpy(np.nonzero(ids == u)[0]).cuda()) for u in range(n) if (ids == u).any()]
        if own:  # the tenants' serving layout and their device table, made once per tenant
            bd = _bd()
            mode, g = (bd.BD_SCALE_GROUP, 128) if case["scales"] == "group" else (bd.BD_SCALE_ROW, 0)
            recs = []
            for sg, sc in zip(st["signs"], st["scales"]):
                so, sco = bd.bd_prepare_tenant(sg, sc, mode, g, rows, cols)
                recs.append((so, sco, mode, g, bd.BD_LAYOUT_TILED))
            st["table"] = bd.TenantTable(recs, "cuda")
    return st


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------
def _pow2(k, dtype=torch.float32):
    """2^k for whole k in the type's normal range (float64: any k used here), from its bits."""
    p = ((k.long() + 1023) << 52).view(torch.float64)
    return p if dtype == torch.float64 else p.to(dtype)


def _quantise(x, fmt):
    """(values on the E2M1 grid, block scales as values, row scales) of a matrix."""
    v = x.float()
    rows, cols = v.shape
    row = torch.ones(rows, device=v.device)
    if fmt == "nv":
        # the least power of two r with max|x| <= 6 * 448 * r; 2688 = 0.65625 * 2^12
        m, e = torch.frexp(v.abs().amax(1))
        k = torch.where(m <= 0.65625, e - 12, e - 11).clamp(-126, 126)
        k = torch.where(m == 0, torch.zeros_like(k), k)
        row = _pow2(k)
        v = v * _pow2(-k)[:, None]
    b = v.view(rows, cols // BLOCK[fmt], BLOCK[fmt])
    top = b.abs().amax(2)
    if fmt == "nv":
        s = (top / 6.0).to(torch.float8_e4m3fn).float()
        q = torch.where(s[:, :, None] > 0, b / s.clamp(min=2.0 ** -9)[:, :, None], torch.zeros_like(b))
    else:
        x2 = torch.where(top > 0, torch.frexp(top)[1] - 3, torch.full_like(top, -127).int()).clamp(-127, 127)
        q = (b.double() * _pow2(-x2, torch.float64)[:, :, None]).float()
        s = _pow2(x2)
    a = q.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign(torch.round(a / step) * step, q)
    return q.view(rows, cols), s, row


def _pack(q):
    """Values on the E2M1 grid -> codes, two per byte."""
    a = q.abs()
    c = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c |= torch.signbit(q).to(torch.uint8) << 3
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _tile(s, fmt):
    """Block scales as values -> their bytes in tiles of 128 rows x 4."""
    rows, nb = s.shape
    if fmt == "nv":
        b = s.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        b = (torch.frexp(s)[1] + 126).to(torch.uint8)
    rt, ct = -(-rows // 128), -(-nb // 4)
    full = torch.zeros((rt * 128, ct * 4), dtype=torch.uint8, device=s.device)
    full[:rows, :nb] = b
    return full.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).reshape(rt, ct, 512)


def _values(p, fmt, dtype=torch.float32):
    """The matrix that codes and scales stand for."""
    rows, cols, block = p["rows"], p["cols"], BLOCK[fmt]
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device="cuda")
    q = torch.stack((grid[(p["codes"] & 15).int()], grid[(p["codes"] >> 4).int()]), dim=2).view(rows, cols)
    rt, ct = p["scales"].shape[:2]
    s = p["scales"].view(rt, ct, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, ct * 4)[:rows, : cols // block]
    if fmt == "nv":
        s = s.contiguous().view(torch.float8_e4m3fn).to(dtype)
    else:
        s = _pow2(s.int() - 127, dtype)
    v = (q.view(rows, cols // block, block) * s[:, :, None]).view(rows, cols)
    return v if p["row"] is None else v * p["row"].to(dtype)[:, None]


def _delta(signs, scales, dtype=torch.float32):
    bits = (signs[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    d = (2 * bits - 1).to(dtype).view(signs.shape[0], -1)
    s = scales.to(dtype)
    if s.dim() == 1:
        return d * s[:, None]
    return (d.view(s.shape[0], s.shape[1], -1) * s[:, :, None]).view(d.shape)


def _plain(st):
    case = st["case"]
    fmt = case["fmt"]
    if case["op"] == "quantize":
        q, s, row = _quantise(st["x"], fmt)
        hat = (q.view(*s.shape, BLOCK[fmt]) * s[:, :, None]).view(q.shape) * row[:, None]
        got = {"hat": hat.to(DTYPE[case["hat"]])}
        return got | {"row": row} if fmt == "nv" else got
    w = _values(st["w"], fmt)
    if case["op"] == "dequantize":
        return w.to(DTYPE[case["out"]])
    x = _values(st["x"], fmt) if case["op"] == "matmul" else st["x"].float()
    y = x @ w.t()
    if case["op"] == "apply":
        for u, at in st["tokens_of"]:
            y[at] += x[at] @ _delta(st["signs"][u], st["scales"][u]).t()
    return y.to(DTYPE[case["out"]])


# ---------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------
def _kept(st, name, make):
    """A buffer that a program keeps from call to call (workspace, outputs)."""
    if name not in st["keep"]:
        st["keep"][name] = make()
    return st["keep"][name]


def _framework(st):
    bd, case = _bd(), st["case"]
    fmt = _fmt(case)
    if case["op"] == "quantize":
        buf = _kept(st, "out", lambda: bd.fp4_buffers(case["rows"], case["cols"], fmt, "cuda"))
        hat = _kept(st, "hat", lambda: torch.empty((case["rows"], case["cols"]), dtype=DTYPE[case["hat"]], device="cuda"))
        bd.bd_quantize_fp4(st["x"], fmt, *buf, hat=hat)
        return {"hat": hat, "row": buf[2]} if case["fmt"] == "nv" else {"hat": hat}
    w = st["w"]
    dt = DTYPE[case["out"]]
    if case["op"] == "dequantize":
        out = _kept(st, "out", lambda: torch.empty((w["rows"], w["cols"]), dtype=dt, device="cuda"))
        return bd.bd_dequantize_fp4(w["codes"], w["scales"], w["row"], fmt, out=out)
    x, t = st["x"], case["tokens"]
    y = _kept(st, "y", lambda: torch.empty((t, w["rows"]), dtype=dt, device="cuda"))
    if case["op"] == "matmul":
        ws = _kept(st, "ws", lambda: bd.fp4_workspace(bd.bd_matmul_fp4_workspace_size(w["rows"], w["cols"], t), "cuda"))
        return bd.bd_matmul_fp4(w["codes"], w["scales"], w["row"], x["codes"], x["scales"], x["row"], fmt, y=y,
                                workspace=ws)[0]
    if case["op"] == "linear":
        ws = _kept(st, "ws", lambda: bd.fp4_workspace(bd.bd_linear_fp4_workspace_size(w["rows"], w["cols"], t), "cuda"))
        return bd.bd_linear_fp4(w["codes"], w["scales"], w["row"], x, fmt, y=y, workspace=ws)[0]
    ws = _kept(st, "ws", lambda: bd.fp4_workspace(
        bd.bd_apply_fp4_workspace_size(w["rows"], w["cols"], t, case["tenants"]), "cuda"))
    return bd.bd_apply_multi_fp4(w["codes"], w["scales"], w["row"], st["table"], st["ids"], x, fmt, y=y, workspace=ws)[0]


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _two_to(k):
    """2^k in 64 bits, by table."""
    return torch.tensor([math.ldexp(1.0, i) for i in range(-260, 261)], dtype=torch.float64, device="cuda")[k.long() + 260]


def _exact_matrix(codes, scales, row, rows, cols, fmt):
    """Each value from its own nibble and its own scale byte, in 64 bits, on the GPU."""
    block = BLOCK[fmt]
    r = torch.arange(rows, device="cuda")[:, None]
    c = torch.arange(cols, device="cuda")[None, :]
    n = (codes[r, c // 2].long() >> (4 * (c % 2))) & 15
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _two_to(e - 1)) * (1 - 2 * (n >> 3)).double()
    b = torch.arange(cols // block, device="cuda")[None, :]
    s = scales[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4].long()
    if fmt == "nv":
        e, m = s >> 3, (s & 7).double()
        s = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _two_to(e - 7))
    else:
        s = _two_to(s - 127)
    v = v * s.repeat_interleave(block, dim=1)
    return v if row is None else v * row.double()[:, None]


def _exact_rows(p, r0, r1, fmt):
    """Rows r0..r1 (r0 a multiple of 128) of a packed matrix."""
    return _exact_matrix(p["codes"][r0:r1], p["scales"][r0 // 128: -(-r1 // 128)],
                         None if p["row"] is None else p["row"][r0:r1], r1 - r0, p["cols"], fmt)


def _nearest(v, grid):
    """The nearest entry of a sorted grid, ties to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    up = torch.bucketize(v, mid)            # values on a border go down here
    tie = torch.zeros_like(up, dtype=torch.bool)
    tie |= v == mid[up.clamp(max=mid.numel() - 1)]
    return grid[torch.where(tie & (up % 2 == 1), up + 1, up)]


def _exact_quantise(x, fmt):
    x = x.double()
    rows, cols = x.shape
    block = BLOCK[fmt]
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    row = torch.ones(rows, dtype=torch.float64, device="cuda")
    if fmt == "nv":
        top = x.abs().amax(1)
        k = torch.ceil(torch.log2(top / 2688)).clamp(-126, 126)
        k += ((top > 2688 * _two_to(k)) & (k < 126)).double()  # (the logarithm is rounded)
        k -= ((top <= 2688 * _two_to(k - 1)) & (k > -126)).double()
        row = torch.where(top > 0, _two_to(k), row)
    v = (x / row[:, None]).view(rows, cols // block, block)
    top = v.abs().amax(2)
    if fmt == "nv":
        code = torch.arange(127, device="cuda")
        e, m = code >> 3, (code & 7).double()
        s = _nearest(top / 6, torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _two_to(e - 7)))
    else:
        lo = torch.floor(torch.log2(top.clamp(min=2.0 ** -200)))
        lo += (_two_to(lo + 1) <= top).double()
        lo -= (_two_to(lo) > top).double()
        s = _two_to((lo - 2).clamp(-127, 127))
    a = torch.where(s[:, :, None] > 0, v.abs() / s.clamp(min=2.0 ** -200)[:, :, None], torch.zeros_like(v))
    hat = torch.sign(v) * _nearest(a, e2m1) * s[:, :, None] * row[:, None, None]
    return hat.view(rows, cols), row


def exact(case, seed):
    st = prepare(case, seed)
    fmt, rows = case["fmt"], case["rows"]
    if case["op"] == "quantize":
        parts = [_exact_quantise(st["x"][r0: r0 + 4096], fmt) for r0 in range(0, rows, 4096)]
        got = {"hat": torch.cat([p[0] for p in parts])}
        return got | {"row": torch.cat([p[1] for p in parts])} if fmt == "nv" else got
    if case["op"] == "dequantize":
        return torch.cat([_exact_rows(st["w"], r0, min(rows, r0 + 4096), fmt) for r0 in range(0, rows, 4096)])
    t = case["tokens"]
    if case["op"] == "matmul":
        x = torch.cat([_exact_rows(st["x"], r0, min(t, r0 + 4096), fmt) for r0 in range(0, t, 4096)])
    else:
        x = st["x"].double()
    y = torch.cat([x @ _exact_rows(st["w"], r0, min(rows, r0 + 4096), fmt).t() for r0 in range(0, rows, 4096)], dim=1)
    if case["op"] == "apply":
        ids = st["ids"].tolist()
        for u in sorted(set(ids) - {-1}):
            at = [i for i, v in enumerate(ids) if v == u]
            words = st["signs"][u].long()
            col = torch.arange(case["cols"], device="cuda")
            sign = ((words[:, col // 32] >> (col % 32)) & 1).double() * 2 - 1
            sc = st["scales"][u].double()
            sign *= sc[:, None] if sc.dim() == 1 else sc[:, col // 128]
            y[at] += x[at] @ sign.t()
    return y
