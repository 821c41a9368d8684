"""The 4-bit wrappers on a stream that is not the current one: what a call allocates belongs to
the stream that it launches on."""

import numpy as np
import pytest

import oracle as O
from helpers import dev
from test_fp4_gpu import _packed, _table
from workloads import activations, random_tenant

pytestmark = pytest.mark.gpu
BUSY = 300_000_000  # cycles, about 0.15 s


@pytest.fixture(scope="module")
def bd():
    from tenant_serving_b200 import build
    build.build()
    import tenant_serving_b200 as m
    return m


def _used(nbytes):
    """Leaves a freed block of ones in the current stream's pool, for the next allocation."""
    import torch
    t = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del t


def test_status_of_a_product_on_another_stream(bd):
    """The current stream is busy: the status word of a workspace that the call made is zeroed on
    the call's stream, before its kernel."""
    import torch
    rng = np.random.default_rng(1)
    w, _ = _packed(bd, rng, 130, 256, O.FP4_NV)
    x, _ = _packed(bd, rng, 7, 256, O.FP4_NV)
    y = torch.empty((7, 130), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    _used(bd.bd_matmul_fp4_workspace_size(130, 256, 7))
    torch.cuda._sleep(BUSY)
    _, ws = bd.bd_matmul_fp4(*w, *x, O.FP4_NV, y=y, stream=side)
    assert bd.bd_get_status(ws, side) == (bd.BD_OK, 0)
    assert not torch.cuda.current_stream().query()  # (it was busy all along)
    torch.cuda.synchronize()
    assert bd.bd_get_status(ws, side) == (bd.BD_OK, 0)


def _calls(bd):
    rng = np.random.default_rng(2)
    w, _ = _packed(bd, rng, 300, 2048, O.FP4_NV)
    x = dev(activations(rng, 70, 2048))
    table = _table(bd, [random_tenant(rng, 300, 2048, 1)])
    ids = dev(np.zeros(70, dtype=np.int32))
    return {
        "quantize": lambda s: bd.bd_quantize_fp4(x, O.FP4_NV, hat_dtype=x.dtype, stream=s),
        "dequantize": lambda s: bd.bd_dequantize_fp4(*w, O.FP4_NV, stream=s),
        "prepare": lambda s: bd.bd_prepare_fp4_scales(w[1].view(-1)[: 300 * 128].view(300, 128), O.FP4_NV, 300, 2048,
                                                     stream=s),
        "matmul": lambda s: bd.bd_matmul_fp4(*w, w[0][:128], w[1][:1], w[2][:128], O.FP4_NV, stream=s),
        "linear": lambda s: bd.bd_linear_fp4(*w, x, O.FP4_NV, stream=s),
        "apply": lambda s: bd.bd_apply_multi_fp4(*w, table, ids, x, O.FP4_NV, stream=s),
    }


@pytest.mark.parametrize("name", ["quantize", "dequantize", "prepare", "matmul", "linear", "apply"])
def test_dropped_results_of_another_stream(bd, name):
    """What a call on a busy side stream returned is dropped before its kernels have run: the
    current stream's next tensors do not get that memory."""
    import torch
    call = _calls(bd)[name]
    side = torch.cuda.Stream()
    sizes = [t.nbytes for t in _flat(call(None))]  # (also loads what a first call loads)
    _used(16)
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = call(side)
    del got
    mine = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.current_stream().synchronize()
    assert not side.query()  # (its kernels are still to come)
    torch.cuda.synchronize()
    assert all(bool((m == 0xA5).all()) for m in mine)


def _flat(r):
    return [t for t in (r if isinstance(r, (tuple, list)) else (r,)) if t is not None]
