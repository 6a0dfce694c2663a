"""A row whose kept tokens are all pinned writes into no block: who else holds
those blocks does not matter to it (kvq_evict_tokens, and the oracle)."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl

# keep, recent, pinned, and whether something below keep is written: a window
# that moves down or a place that may be filled
CASES = [(40, 0, 40, False), (40, 0, 2 ** 31 - 1, False), (33, 0, 33, False), (48, 0, 48, False), (0, 0, 0, False),
         (0, 5, 7, False), (40, 0, 39, True), (40, 1, 40, True), (40, 40, 40, True), (33, 0, 32, True)]


def _refs(nb, table, keep):
    """Every block of the row's first keep tokens is held by another row, too."""
    refs = np.ones(nb, np.int64)
    refs[table[:-(-keep // 16)]] = 2
    return refs


@pytest.mark.parametrize("keep,recent,pinned,writes", CASES)
def test_oracle(keep, recent, pinned, writes):
    codes = np.arange(9 * 16 * 2).reshape(9, 16, 2)
    weights = np.random.default_rng(keep).random((1, 2, 128)).astype(np.float32)
    table = np.random.default_rng(1).permutation(9)[:7]
    before, old = codes.copy(), weights.copy()
    kept = oracle.evict_tokens([keep], [recent], [pinned], [100], table[None], [codes], weights, _refs(9, table, keep))
    assert kept.tolist() == [100 if writes else keep]
    assert (codes == before).all()
    if not writes:
        old[:, :, keep:100] = 0
    assert (weights == old).all()


@pytest.mark.gpu
@pytest.mark.parametrize("keep,recent,pinned,writes", CASES)
def test_kernel(keep, recent, pinned, writes):
    from quantized_paged_kv_write_gb300 import build
    build.build()
    import quantized_paged_kv_write_gb300 as kvq
    f = wl.CacheFormat(wl.INT8, wl.PER_TOKEN_HEAD)
    fmt = kvq.cache_format(f, f, 2, 64, 9)
    cache = kvq.allocate_cache(fmt)
    gen = torch.Generator(device="cuda").manual_seed(2)
    for x in cache.values():
        x.copy_(torch.randint(0, 256, x.shape, generator=gen, device="cuda"))
    weights = torch.rand((1, 2, 128), generator=gen, device="cuda")
    table = np.random.default_rng(1).permutation(9)[:7]
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    before, old = {k: x.clone() for k, x in cache.items()}, weights.clone()
    kept = kvq.kvq_evict_tokens(i32([keep]), i32([100]), i32(table[None]), fmt, cache, weights, i32([recent]),
                                pinned_lens=i32([pinned]), pool=dict(ref_counts=i32(_refs(9, table, keep))))
    assert kvq.kvq_device_errors() == (kvq.DEVERR_POOL_STATE if writes else 0)
    assert kept.tolist() == [100 if writes else keep]
    assert all(torch.equal(before[k], x) for k, x in cache.items())
    if not writes:
        old[:, :, keep:100] = 0
    assert torch.equal(weights, old)
