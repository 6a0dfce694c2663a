"""kvq_assign_blocks / kvq_release_blocks against the oracle's loops
(oracle/block_pool.py): every output and the whole state, value for value."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

kvq = None


@pytest.fixture(scope="module", autouse=True)
def _lib():
    global kvq
    from quantized_paged_kv_write_gb300 import build
    build.build()
    import quantized_paged_kv_write_gb300 as m
    m.load_library()
    kvq = m
    yield
    assert kvq.kvq_device_errors() == 0


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Both:
    """The same state on the device and in the oracle."""

    def __init__(self, rows, width, nb, seed=0):
        self.rng = np.random.default_rng(seed)
        order = self.rng.permutation(nb)
        self.pool = oracle.Pool(order, nb)
        self.ctx, self.tables = np.zeros(rows, np.int64), np.full((rows, width), -1)
        self.dpool = kvq.allocate_pool(nb)
        self.dpool["free_list"].copy_(_i32(order))
        self.dctx, self.dtables = _i32(self.ctx), _i32(self.tables)

    def assign(self, n, cap=None, rows=None, blocks=None):
        cap = int(sum(n)) + 3 if cap is None else cap
        want = oracle.assign_blocks(self.pool, n, self.ctx, self.tables, cap, rows, blocks)
        got = kvq.kvq_assign_blocks(_i32(n), self.dctx, self.dtables, self.dpool, cap,
                                    prefix_rows=None if rows is None else _i32(rows),
                                    prefix_blocks=None if blocks is None else _i32(blocks))
        for g, w, what in zip(got, want[1:], ("offsets", "slots", "positions")):
            assert np.array_equal(g.cpu().numpy(), w), what
        self.check()
        return want[0]

    def release(self, keep):
        oracle.release_blocks(self.pool, keep, self.ctx, self.tables)
        kvq.kvq_release_blocks(_i32(keep), self.dctx, self.dtables, self.dpool)
        self.check()

    def check(self):
        assert np.array_equal(self.dctx.cpu().numpy(), self.ctx)
        assert np.array_equal(self.dtables.cpu().numpy(), self.tables)
        n = int(self.dpool["free_count"])
        assert n == len(self.pool.free)
        assert self.dpool["free_list"][:n].cpu().tolist() == self.pool.free
        assert np.array_equal(self.dpool["ref_counts"].cpu().numpy(), self.pool.refs)


@pytest.mark.parametrize("rows,width,nb,most", [
    (1, 1, 1, 16), (1, 40, 30, 200), (2, 5, 9, 40), (31, 7, 100, 60), (33, 20, 300, 90), (257, 9, 1200, 40),
    (1025, 6, 4000, 30), (64, 300, 9000, 2000)])
def test_random_runs(rows, width, nb, most):
    s = Both(rows, width, nb, seed=rows)
    done = 0
    for step in range(12):
        room = width * 16 - s.ctx
        n = np.minimum(s.rng.integers(0, most + 1, rows) * (s.rng.random(rows) < 0.7), room)
        while (-(-(s.ctx + n) // 16) - -(-s.ctx // 16)).sum() > len(s.pool.free):
            n = n // 2
        assert s.assign(n)
        done += int(n.sum())
        if step % 3 == 2:
            s.release(s.rng.integers(0, width * 20, rows) * (s.rng.random(rows) < 0.8))
    assert done > 0


def test_shared_prefixes_come_and_go():
    s = Both(40, 70, 700, seed=5)
    n = np.zeros(40, int)
    n[39] = 50 * 16 + 3                              # the row that keeps the prompt
    assert s.assign(n)
    rows, blocks = np.full(40, -1), np.zeros(40, int)
    rows[:30], blocks[:30] = 39, s.rng.integers(0, 51, 30)
    n = s.rng.integers(0, 40, 40)
    n[39] = 0
    assert s.assign(n, rows=rows, blocks=blocks)
    s.release(np.where(np.arange(40) < 15, 0, 5000))  # half the readers leave
    s.release(np.where(np.arange(40) == 39, 0, 5000))  # the keeper leaves: the rest still hold the blocks
    rows[:], blocks[:] = -1, 0
    big = int(np.argmax(np.where(np.arange(40) < 30, s.ctx, -1)))
    rows[0], blocks[0] = big, s.ctx[big] // 16        # share from a row that shares itself
    n[:] = 1
    n[0] = 20
    part = (s.ctx % 16 != 0) & (s.pool.refs[np.maximum(s.tables[np.arange(40), np.minimum(s.ctx // 16, 69)], 0)] > 1)
    n[part] = 0
    assert s.assign(n, rows=rows, blocks=blocks)
    s.release(np.zeros(40, int))                      # all at once, shared blocks by several rows
    assert len(s.pool.free) == 700


@pytest.mark.parametrize("rows,shared,keepers", [(2, 40, 1), (9, 33, 1), (16, 300, 2), (67, 129, 3), (24, 2100, 1),
                                                 (530, 2048, 1)])
def test_long_rows_behind_shared_prefixes(rows, shared, keepers):
    """Rows of one id per column next to rows of others, ends and beginnings in
    the middle of the shared blocks; the largest has more items than a warp's
    first 64 turns hold."""
    width, live = shared + 6, rows - keepers
    s = Both(rows, width, keepers * shared + live * 7 + 3, seed=rows + shared)
    n = np.zeros(rows, int)
    n[live:] = shared * 16                               # the prompts
    assert s.assign(n)
    src, blocks = np.full(rows, -1), np.zeros(rows, int)
    src[:live] = live + np.sort(s.rng.integers(0, keepers, live))
    blocks[:live] = np.where(s.rng.random(live) < 0.7, shared, s.rng.integers(0, shared + 1, live))
    n = np.where(np.arange(rows) < live, s.rng.integers(0, 90, rows), 0)
    assert s.assign(n, rows=src, blocks=blocks)
    some = s.rng.random(rows) < 0.5
    s.release(np.where(some, s.rng.integers(0, shared * 16, rows) // 16 * 16, 10 ** 6))  # back into the shared blocks
    s.release(np.where(s.rng.random(rows) < 0.3, 0, 10 ** 6))
    s.release(np.zeros(rows, int))                       # all at once
    assert len(s.pool.free) == len(s.pool.refs)


def test_a_captured_admission_with_many_shared_blocks():
    """The largest clusters in a graph: admit and evict, replayed."""
    rows, shared = 65, 2048
    s = Both(rows, shared + 10, shared + 64 * 9 + 5, seed=21)
    assert s.assign([0] * 64 + [shared * 16])
    n, keep = _i32([100] * 64 + [0]), _i32([0] * 64 + [10 ** 6])
    src, blocks = _i32([64] * 64 + [-1]), _i32([shared] * 64 + [0])
    before = {k: v.clone() for k, v in s.dpool.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kvq.kvq_assign_blocks(n, s.dctx, s.dtables, s.dpool, 6400, prefix_rows=src, prefix_blocks=blocks)
        held = s.dpool["ref_counts"].clone()
        kvq.kvq_release_blocks(keep, s.dctx, s.dtables, s.dpool)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        s.check()                                         # the pool and tables are as they were
        assert torch.equal(s.dpool["free_list"], before["free_list"])
        ids = s.dtables[64, :shared].long()
        assert (held[ids] == 65).all() and int(held.sum()) == 65 * shared + 64 * 7
        assert int(out[0][-1]) == 6400 and int(out[1].min()) >= 0
        for x in out:
            x.zero_()


def test_more_given_back_than_held():
    """Tables that list a block more often than its count says: the block goes
    back once, the counts end at 0, the bit is set."""
    for rows, width in ((3, 4), (20, 64)):               # by items and by columns
        pool = kvq.allocate_pool(width)
        pool["free_count"].zero_()
        pool["ref_counts"].fill_(2)
        tables = _i32(np.tile(np.arange(width), (rows, 1)))
        tables[0, 0] = -7
        ctx = _i32([16 * width] * rows)
        kvq.kvq_release_blocks(_i32([0] * rows), ctx, tables, pool)
        assert kvq.kvq_device_errors() == kvq.DEVERR_POOL_STATE | kvq.DEVERR_BLOCK_RANGE
        assert (tables == -1).all() and (pool["ref_counts"] == 0).all() and (ctx == 0).all()
        assert int(pool["free_count"]) == width
        assert sorted(pool["free_list"].tolist()) == list(range(width))


def test_release_undoes_assign_exactly():
    s = Both(50, 30, 900, seed=6)
    assert s.assign(s.rng.integers(0, 200, 50))
    free, ctx = list(s.pool.free), s.ctx.copy()
    assert s.assign(s.rng.integers(0, 100, 50))
    s.release(ctx)
    assert s.pool.free == free


def test_capacity_and_range_errors_change_nothing():
    s = Both(4, 8, 10, seed=7)
    assert s.assign([20, 0, 5, 0])
    full = dict(rows=[-1, 0, -1, -1], blocks=[0, 1, 0, 0])
    for n, kw, bit in [
            ([200, 0, 0, 0], {}, kvq.DEVERR_CONTEXT_RANGE),           # past the table
            ([100, 60, 0, 0], {}, kvq.DEVERR_CAPACITY),               # more blocks than free
            ([3, 0, 4, 0], dict(cap=6), kvq.DEVERR_CAPACITY),         # more tokens than room
            ([1, -1, 0, 0], {}, kvq.DEVERR_CONTEXT_RANGE),
            ([0, 1, 0, 0], dict(rows=[-1, 0, -1, -1], blocks=[0, 2, 0, 0]), kvq.DEVERR_CONTEXT_RANGE),  # not full yet
            ([0, 1, 0, 0], dict(rows=[-1, 1, -1, -1], blocks=[0, 0, 0, 0]), kvq.DEVERR_CONTEXT_RANGE),  # itself
            ([0, 1, 0, 0], dict(rows=[-1, 9, -1, -1], blocks=[0, 0, 0, 0]), kvq.DEVERR_CONTEXT_RANGE),
            ([0, 1, 0, 0], dict(rows=[1, -1, -1, -1], blocks=[0, 0, 0, 0]), kvq.DEVERR_CONTEXT_RANGE)]:  # not empty
        assert not s.assign(n, **kw), (n, kw)
        assert kvq.kvq_device_errors() == bit, (n, kw)
    assert s.assign([0, 3, 0, 0], **full)
    s.release([9, 5000, 5000, 5000])                  # row 0 ends inside the block that row 1 shares
    assert not s.assign([1, 0, 0, 0])                 # and may not write into it
    assert kvq.kvq_device_errors() == kvq.DEVERR_POOL_STATE
    s.release([-1, 5000, 0, 0])
    assert kvq.kvq_device_errors() == kvq.DEVERR_CONTEXT_RANGE


def test_a_block_given_back_twice_is_refused():
    s = Both(2, 4, 6, seed=8)
    assert s.assign([16, 16])
    s.tables[1, 0] = s.tables[0, 0]                   # a table that the calls did not make
    s.dtables.copy_(_i32(s.tables))
    s.release([0, 0])
    assert kvq.kvq_device_errors() == kvq.DEVERR_POOL_STATE


def test_bad_table_entries_are_cleared():
    s = Both(2, 4, 6, seed=9)
    assert s.assign([40, 5])
    s.tables[0, 1], s.tables[0, 2] = 99, -7
    s.dtables.copy_(_i32(s.tables))
    s.release([0, 0])
    assert kvq.kvq_device_errors() == kvq.DEVERR_BLOCK_RANGE


def test_no_rows_and_the_most_rows():
    pool = kvq.allocate_pool(3)
    z, t = _i32(np.zeros(0)), torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    off, slots, pos = kvq.kvq_assign_blocks(z, z, t, pool, 4)
    assert off.tolist() == [0] and slots.tolist() == [-1] * 4 and pos.tolist() == [-1] * 4
    kvq.kvq_release_blocks(z, z, t, pool)
    s = Both(8192, 2, 9000, seed=10)
    assert s.assign(s.rng.integers(0, 17, 8192))
    assert s.assign(np.minimum(1, 32 - s.ctx))
    s.release(s.rng.integers(0, 20, 8192))


def test_a_captured_step_replays_and_streams():
    # one token a row and step, with a rollback of every third row's step
    s = Both(20, 30, 400, seed=11)
    assert s.assign(s.rng.integers(1, 100, 20))
    n, cap = _i32(np.ones(20)), 20
    off = torch.empty(21, dtype=torch.int32, device="cuda")
    slots, pos = torch.empty(cap, dtype=torch.int64, device="cuda"), torch.empty(cap, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kvq.kvq_assign_blocks(n, s.dctx, s.dtables, s.dpool, cap, token_offsets=off, slot_mapping=slots, positions=pos)
    for step in range(40):
        graph.replay()
        ok, w_off, w_slots, w_pos = oracle.assign_blocks(s.pool, np.ones(20, int), s.ctx, s.tables, cap)
        assert ok and slots.tolist() == w_slots.tolist() and pos.tolist() == w_pos.tolist(), step
        s.check()
        if step % 3 == 0:
            s.release(np.where(np.arange(20) % 3 == 0, s.ctx - 1, 10_000))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    kvq.kvq_assign_blocks(n, s.dctx, s.dtables, s.dpool, cap, stream=other)
    other.synchronize()
    oracle.assign_blocks(s.pool, np.ones(20, int), s.ctx, s.tables, cap)
    s.check()
