"""kvq_assign_blocks on states that it must refuse as a whole: nothing changes,
on any of the cluster's CTAs."""
import numpy as np
import pytest
import torch

from tests import test_gpu_block_pool as base

pytestmark = pytest.mark.gpu

kvq = None


@pytest.fixture(scope="module", autouse=True)
def _lib():
    global kvq
    from quantized_paged_kv_write_gb300 import build
    build.build()
    import quantized_paged_kv_write_gb300 as m
    m.load_library()
    kvq = base.kvq = m
    yield
    assert kvq.kvq_device_errors() == 0


def _behind_a_prompt(rows, shared, seed):
    """`rows` empty rows and one that holds `shared` full blocks."""
    s = base.Both(rows + 1, shared + 8, shared + rows * 8 + 5, seed=seed)
    n = np.zeros(rows + 1, int)
    n[rows] = shared * 16
    assert s.assign(n)
    src, blocks = np.full(rows + 1, rows), np.full(rows + 1, shared)
    src[rows], blocks[rows] = -1, 0
    return s, src, blocks


@pytest.mark.parametrize("rows,shared", [(1, 3), (9, 40), (64, 2048)])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])
def test_a_bad_block_in_the_shared_part_changes_nothing(rows, shared, bad):
    s, src, blocks = _behind_a_prompt(rows, shared, 41)
    for at in (0, shared // 2, shared - 1):
        kept = s.tables[rows, at]
        s.tables[rows, at] = bad
        s.dtables.copy_(base._i32(s.tables))
        n = np.arange(rows + 1) % 60 * (np.arange(rows + 1) < rows)
        assert not s.assign(n, rows=src, blocks=blocks)
        assert kvq.kvq_device_errors() == kvq.DEVERR_BLOCK_RANGE
        if at > 0:                                       # the rows stop short of it
            assert s.assign(0 * n, rows=src, blocks=np.minimum(blocks, at))
            s.release(np.where(np.arange(rows + 1) < rows, 0, 10 ** 6))
        s.tables[rows, at] = kept
        s.dtables.copy_(base._i32(s.tables))
    assert s.assign(n, rows=src, blocks=blocks)


@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31])
def test_a_bad_free_block_changes_nothing(bad):
    for rows, tokens in ((3, 20), (64, 4097)):           # one CTA, many
        s = base.Both(rows, tokens // 16 + 2, rows * (tokens // 16 + 2), seed=42)
        at = len(s.pool.free) - 1 - rows * (tokens // 16 + 1) // 2
        kept, s.pool.free[at] = s.pool.free[at], bad
        s.dpool["free_list"][at] = bad
        assert not s.assign([tokens] * rows)
        assert kvq.kvq_device_errors() == kvq.DEVERR_POOL_STATE
        if rows > 3:
            assert s.assign([16] * rows)                 # stops before the bad entry
        s.pool.free[at] = kept
        s.dpool["free_list"][at] = kept
        assert s.assign([tokens - 16] * rows)


def test_every_cta_comes_to_the_same_verdict():
    """A pool whose counts miss a user of a block: the check sees the counts from
    before the call on every CTA, so the whole call is done (or none of it)."""
    rows, shared = 64, 2048
    for attempt in range(20):
        s, src, blocks = _behind_a_prompt(rows, shared, 43 + attempt)
        # the last row of the readers continues a block that the prompt lists too
        src[rows - 1], blocks[rows - 1] = -1, 0
        s.ctx[rows - 1] = 5
        s.tables[rows - 1, 0] = s.tables[rows, 7]
        s.dctx.copy_(base._i32(s.ctx))
        s.dtables.copy_(base._i32(s.tables))
        n = np.full(rows + 1, 40)
        n[rows] = 0
        assert s.assign(n, rows=src, blocks=blocks)
        assert kvq.kvq_device_errors() == 0
