"""Decodes of fewer blocks than the launch has CTAs for (contexts far below
max_context_len, or one long one among short ones): every partial that the
reduce reads has to be the call's own, whatever the workspace held before."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from tests._helpers import bits, check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("contexts,longest", [([33], 4096), ([0, 1, 15, 16, 17, 300, 33, 1000, 0], 1000),
                                              ([40, 70, 5], 30000), ([2000], 60000)])
@pytest.mark.parametrize("stale", [0.0, 50.0])
@pytest.mark.parametrize("tail", [False, True])
def test_stale_partials_are_not_read(contexts, longest, stale, tail):
    from quantized_paged_kv_write_gb300 import build
    build.build()
    import quantized_paged_kv_write_gb300 as kvq
    k = wl.CacheFormat(wl.INT8, wl.PER_BLOCK_CHANNEL if tail else wl.PER_TOKEN_HEAD)
    v = wl.CacheFormat(wl.INT8, wl.PER_TOKEN_HEAD)
    if tail:
        contexts = [n // 16 * 16 for n in contexts]          # (complete blocks: the tail is empty)
    b, held = len(contexts), [-(-n // 16) for n in contexts]
    nb, width = sum(held), -(-longest // 16)
    fmt = kvq.cache_format(k, v, 2, 64, nb)
    cache, oc = kvq.allocate_cache(fmt), oracle.OracleCache(nb, 16, 2, 64, k, v)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2, nb * 16, 2, 64), generator=gen, device="cuda").to(torch.bfloat16)
    slots = torch.arange(nb * 16, device="cuda")
    kvq.kvq_quantize_write(x[0], x[1], slots, fmt, cache)
    oracle.quantize_write(oc, bits(x[0]), bits(x[1]), slots.cpu().numpy())
    tables, at = np.full((b, width), -1, np.int32), 0
    for r, h in enumerate(held):
        tables[r, :h] = np.arange(at, at + h)
        at += h
    q = torch.randn((b, 4, 64), generator=gen, device="cuda").to(torch.bfloat16)
    t, c = torch.from_numpy(tables).cuda(), torch.tensor(contexts, dtype=torch.int32, device="cuda")
    ws = torch.full((kvq.kvq_decode_workspace_size(fmt, b, 4, longest) // 4 + 64,), stale, device="cuda").view(torch.uint8)
    if tail:
        out = kvq.kvq_kivi_decode(q, fmt, cache, t, c, longest, kvq.allocate_residual(fmt, b), workspace=ws)
    else:
        out = kvq.kvq_paged_decode(q, fmt, cache, t, c, longest, workspace=ws)
    check_attention(out.cpu().numpy(), oracle.paged_decode_fp64(oc, bits(q), tables, contexts), str(contexts))
    assert kvq.kvq_device_errors() == 0
