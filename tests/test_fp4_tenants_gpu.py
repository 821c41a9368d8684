"""Tenants over a 4-bit base in the forms that bd_apply_multi takes them: from the host-resident
cache, with fp32 scales, and the same call again with other tenants in a captured graph."""

import numpy as np
import pytest

import oracle as O
from helpers import assert_apply_close, dev, host
from test_fp4_gpu import _packed, _table
from workloads import activations, random_tenant

pytestmark = pytest.mark.gpu
FMTS = [O.FP4_NV, O.FP4_MX]


@pytest.fixture(scope="module")
def bd():
    from tenant_serving_b200 import build
    build.build()
    import tenant_serving_b200 as m
    return m


@pytest.mark.parametrize("fmt", FMTS)
def test_tenants_of_a_cache(bd, fmt):
    import torch
    d_out, d_in, n_host, n_slots = 700, 640, 7, 3
    rng = np.random.default_rng(4)
    cache = bd.TenantCache([(d_out, d_in, 64)], n_host_tenants=n_host, n_slots=n_slots, device="cuda")
    ten, keep = [], []
    for u, (mode, g) in enumerate([(0, 128), (1, 0), (0, 64), (2, 0), (3, 0), (0, 128), (1, 0)]):
        t = random_tenant(rng, d_out, d_in, mode, g or 128)
        keep.append(bd.bd_prepare_record_host(t["signs"], t["scales"], mode, t["group_size"], d_out, d_in, pin=True))
        cache.register(u, 0, keep[-1], mode, t["group_size"])
        ten.append(t)
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    copy_s, comp_s = torch.cuda.Stream(), torch.cuda.current_stream()
    for k in range(6):  # consecutive batches share few tenants, so slots are filled again
        ids = rng.choice([k % n_host, (k + 3) % n_host, -1], size=30, p=[0.5, 0.4, 0.1]).astype(np.int32)
        slots, _, ticket = cache.prefetch(ids, stream=copy_s)
        cache.acquire(ticket, stream=comp_s)
        xb = activations(rng, len(ids), d_in)
        y, ws = bd.bd_apply_multi_fp4(*w, cache.table(0), dev(slots), dev(xb), fmt, y_dtype=torch.float32)
        cache.release(ticket, stream=comp_s)
        assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
        assert_apply_close(host(y), O.apply_multi_fp4(*wh, fmt, ten, ids, xb, "bf16"), per_token=True)
    torch.cuda.synchronize()
    cache.close()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d_out,d_in", [(300, 512), (40, 96)])
def test_tenants_with_fp32_scales(bd, fmt, d_out, d_in):
    import torch
    rng = np.random.default_rng(d_in)
    ten = [random_tenant(rng, d_out, d_in, m, g, scale_dtype="f32") for m, g in [(0, 32), (1, 0), (2, 0), (3, 0)]]
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    ids = rng.integers(-1, 4, size=50).astype(np.int32)
    xb = activations(rng, 50, d_in)
    y, ws = bd.bd_apply_multi_fp4(*w, _table(bd, ten), dev(ids), dev(xb), fmt, y_dtype=torch.float32)
    assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
    assert_apply_close(host(y), O.apply_multi_fp4(*wh, fmt, ten, ids, xb, "bf16"), per_token=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t", [3, 40, 90])
def test_captured_call_with_other_ids(bd, fmt, t):
    """One captured call: other tokens, ids and tenants' counts with every replay."""
    import torch
    rng = np.random.default_rng(t)
    d_out, d_in = 520, 768
    ten = [random_tenant(rng, d_out, d_in, m, g) for m, g in [(0, 128), (1, 0), (4, 256), (2, 0), (0, 32)]]
    table = _table(bd, ten)
    w, wh = _packed(bd, rng, d_out, d_in, fmt)
    x, ids = torch.zeros((t, d_in), dtype=torch.bfloat16, device="cuda"), torch.zeros(t, dtype=torch.int32, device="cuda")
    y = torch.empty((t, d_out), device="cuda")
    ws = bd.fp4_workspace(bd.bd_apply_fp4_workspace_size(d_out, d_in, t, 5), "cuda")
    bd.bd_apply_multi_fp4(*w, table, ids, x, fmt, y=y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bd.bd_apply_multi_fp4(*w, table, ids, x, fmt, y=y, workspace=ws)
    for kind in range(4):
        n = rng.integers(-1, 5, size=t) if kind == 0 else np.full(t, kind - 2)
        n = n.astype(np.int32)
        xb = activations(rng, t, d_in)
        x.copy_(dev(xb))
        ids.copy_(dev(n))
        g.replay()
        assert bd.bd_get_status(ws) == (bd.BD_OK, 0)
        assert_apply_close(host(y), O.apply_multi_fp4(*wh, fmt, ten, n, xb, "bf16"), per_token=True)
