"""The wrappers on a stream that is not the current one: what a call allocates belongs to the
stream that it launches on (the 4-bit ones have a file of their own)."""

import numpy as np
import pytest

from helpers import dev, host
from workloads import activations, random_tenant, weight_pair

pytestmark = pytest.mark.gpu
BUSY = 300_000_000  # cycles, about 0.15 s


@pytest.fixture(scope="module")
def bd():
    from tenant_serving_b200 import build
    build.build()
    import tenant_serving_b200 as m
    return m


def _flat(r):
    return [t for t in (r if isinstance(r, (tuple, list)) else (r,)) if t is not None]


@pytest.mark.parametrize("entry", ["bd_compress", "bd_compress_noalloc"])
def test_statistics_of_another_stream(bd, entry):
    """The current stream is busy: the statistics that a call returns are not zeroed after it has
    written them."""
    import torch
    wb, wf = (dev(w, "bf16") for w in weight_pair(3, 256, 512, "bf16", 0.02, 0.002, 0.001, 20.0))
    cfg = bd.compress_cfg(mode=bd.BD_SCALE_GROUP, group_size=128, clip=True)
    call = getattr(bd, entry)
    want = [host(t) for t in call(wb, wf, cfg)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = call(wb, wf, cfg, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # (it was busy all along)
    torch.cuda.synchronize()
    assert all(np.array_equal(a, host(b)) for a, b in zip(want, got))


def _calls(bd):
    rng = np.random.default_rng(2)
    d_out, d_in = 300, 2048
    wb, wf = (dev(w, "bf16") for w in weight_pair(5, d_out, d_in, "bf16", 0.02, 0.002, 0.001, 20.0))
    cfg = bd.compress_cfg(mode=bd.BD_SCALE_GROUP, group_size=128, clip=True)
    ten = random_tenant(rng, d_out, d_in, 1)
    signs, scales = dev(ten["signs"]), dev(ten["scales"])
    table = bd.TenantTable([(*bd.bd_prepare_tenant(signs, scales, 1, 0, d_out, d_in), 1, 0, bd.BD_LAYOUT_TILED)], "cuda")
    x, ids = dev(activations(rng, 70, d_in)), dev(np.zeros(70, dtype=np.int32))
    q = bd.bd_quantize_base_fp8(wb)
    return {
        "compress": lambda s: bd.bd_compress(wb, wf, cfg, stream=s),
        "compress_noalloc": lambda s: bd.bd_compress_noalloc(wb, wf, cfg, stream=s),
        "reconstruct": lambda s: bd.bd_reconstruct(signs, scales, 1, 0, d_out, d_in, wb, stream=s),
        "prepare": lambda s: bd.bd_prepare_tenant(signs, scales, 1, 0, d_out, d_in, stream=s),
        "apply": lambda s: bd.bd_apply_multi(wb, table, ids, x, stream=s),
        "quantize_fp8": lambda s: bd.bd_quantize_base_fp8(wb, stream=s),
        "apply_fp8": lambda s: bd.bd_apply_multi_fp8(*q, table, ids, x, stream=s),
    }


@pytest.mark.parametrize("name", ["compress", "compress_noalloc", "reconstruct", "prepare", "apply", "quantize_fp8",
                                  "apply_fp8"])
def test_dropped_results_of_another_stream(bd, name):
    """What a call on a busy side stream returned is dropped before its kernels have run: the
    current stream's next tensors do not get that memory."""
    import torch
    call = _calls(bd)[name]
    side = torch.cuda.Stream()
    sizes = [t.nbytes for t in _flat(call(None))]  # (also loads what a first call loads)
    torch.full((16,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
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
