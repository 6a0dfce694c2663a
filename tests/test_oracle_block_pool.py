"""Pins of the oracle's block pool (oracle/block_pool.py): hand cases and
invariants of random runs."""
import numpy as np

import oracle


def test_hand_case():
    pool = oracle.Pool([5, 4, 3, 2, 1, 0], 6)
    ctx, tables = np.array([0, 15]), np.full((2, 3), -1)
    pool.free.remove(4)
    pool.refs[4] = 1
    tables[1, 0] = 4
    ok, off, slots, pos = oracle.assign_blocks(pool, [17, 2], ctx, tables, 20)
    assert ok and list(off) == [0, 17, 19]
    # row 0 takes blocks 0 and 1, row 1 fills block 4 and takes block 2
    assert tables.tolist() == [[0, 1, -1], [4, 2, -1]]
    assert slots.tolist() == list(range(16)) + [16, 4 * 16 + 15, 2 * 16, -1]
    assert pos.tolist() == list(range(17)) + [15, 16, -1]
    assert ctx.tolist() == [17, 17] and pool.free == [5, 3]
    oracle.release_blocks(pool, [1, 17], ctx, tables)
    assert tables.tolist() == [[0, -1, -1], [4, 2, -1]] and pool.free == [5, 3, 1] and ctx.tolist() == [1, 17]


def test_a_shared_block_outlives_its_first_owner():
    pool = oracle.Pool(range(8), 8)
    ctx, tables = np.array([0, 0]), np.full((2, 4), -1)
    assert oracle.assign_blocks(pool, [40, 0], ctx, tables, 40)[0]
    assert oracle.assign_blocks(pool, [0, 3], ctx, tables, 3, [-1, 0], [0, 2])[0]
    assert (tables[1, :2] == tables[0, :2]).all() and ctx.tolist() == [40, 35]
    shared = [int(x) for x in tables[0, :2]]
    oracle.release_blocks(pool, [0, 99], ctx, tables)
    assert not set(shared) & set(pool.free) and (pool.refs[shared] == 1).all()
    oracle.release_blocks(pool, [0, 0], ctx, tables)
    assert sorted(pool.free) == list(range(8)) and not pool.refs.any()


def test_random_runs_never_lose_or_share_a_block_by_mistake():
    rng = np.random.default_rng(3)
    nb, rows, width = 60, 9, 12
    pool = oracle.Pool(rng.permutation(nb), nb)
    ctx, tables = np.zeros(rows, np.int64), np.full((rows, width), -1)
    for _ in range(200):
        if rng.random() < 0.6:
            before = (list(pool.free), ctx.copy(), tables.copy(), pool.refs.copy())
            keep = ctx.copy()
            n = rng.integers(0, 30, rows) * (rng.random(rows) < 0.5)
            if oracle.assign_blocks(pool, n, ctx, tables, 500)[0] and rng.random() < 0.3:
                oracle.release_blocks(pool, keep, ctx, tables)      # undone: all as before
                assert pool.free == before[0] and (pool.refs == before[3]).all()
                assert (ctx == before[1]).all() and (tables == before[2]).all()
        else:
            oracle.release_blocks(pool, rng.integers(0, 200, rows), ctx, tables)
        used = tables[tables >= 0]
        assert len(set(used.tolist())) == len(used) and sorted(used.tolist() + pool.free) == list(range(nb))
        assert (np.bincount(used, minlength=nb) == pool.refs).all()
        assert ((tables >= 0).sum(1) == -(-ctx // 16)).all()


def test_a_bad_entry_in_what_is_shared_or_taken_refuses_the_call():
    for where in ("shared", "free"):
        pool = oracle.Pool(range(8), 8)
        ctx, tables = np.array([0, 0]), np.full((2, 4), -1)
        assert oracle.assign_blocks(pool, [40, 0], ctx, tables, 40)[0]
        if where == "shared":
            tables[0, 1] = 8
        else:
            pool.free[-1] = -3
        before = (list(pool.free), ctx.copy(), tables.copy(), pool.refs.copy())
        ok, off, slots, _ = oracle.assign_blocks(pool, [0, 3], ctx, tables, 3, [-1, 0], [0, 2])
        assert not ok and not off.any() and (slots == -1).all()
        assert pool.free == before[0] and (ctx == before[1]).all() and (tables == before[2]).all()
        assert (pool.refs == before[3]).all()
        if where == "shared":                        # as far as the good entries go
            assert oracle.assign_blocks(pool, [0, 3], ctx, tables, 3, [-1, 0], [0, 1])[0]
