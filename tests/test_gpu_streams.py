"""What a decode allocates for itself belongs to the stream that it runs on."""
import numpy as np
import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("by_handle", [False, True])
def test_decodes_allocate_on_their_own_stream(monkeypatch, by_handle):
    from quantized_paged_kv_write_gb300 import build
    build.build()
    import quantized_paged_kv_write_gb300 as kvq
    f = wl.CacheFormat(wl.INT8, wl.PER_TOKEN_HEAD)
    c = wl.CacheFormat(wl.INT8, wl.PER_BLOCK_CHANNEL)
    fmt, chan = kvq.cache_format(f, f, 2, 128, 8), kvq.cache_format(c, f, 2, 128, 8)
    gen = torch.Generator(device="cuda").manual_seed(0)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    tables = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    ctx = torch.tensor([33, 50], dtype=torch.int32, device="cuda")
    q, k, v = draw(2, 8, 128), draw(2, 2, 128), draw(2, 2, 128)
    cache, ccache, res = kvq.allocate_cache(fmt), kvq.allocate_cache(chan), kvq.allocate_residual(chan, 2)
    kvq.kvq_quantize_write(draw(128, 2, 128), draw(128, 2, 128), torch.arange(128, device="cuda"), fmt, cache)
    kvq.kvq_quantize_write(draw(128, 2, 128), draw(128, 2, 128), torch.arange(128, device="cuda"), chan, ccache)
    calls = [lambda s: kvq.kvq_write_decode(q, k, v, fmt, cache, tables, ctx, 50, stream=s),
             lambda s: kvq.kvq_paged_decode(q, fmt, cache, tables, ctx, 50, stream=s),
             lambda s: kvq.kvq_kivi_decode(q, chan, ccache, tables, ctx, 50, res, stream=s)]
    want = [f(None) for f in calls]
    torch.cuda.synchronize()
    side, plain, where = torch.cuda.Stream(), torch.empty, []

    def empty(*a, **kw):
        where.append(torch.cuda.current_stream().cuda_stream)
        return plain(*a, **kw)
    monkeypatch.setattr(torch, "empty", empty)
    for f, w in zip(calls, want):
        out = f(side.cuda_stream if by_handle else side)
        torch.cuda.synchronize()
        assert torch.equal(out, w) and np.isfinite(out.cpu().numpy()).all()
    assert where == [side.cuda_stream] * 6
