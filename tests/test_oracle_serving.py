"""Pins of the oracle's prompt attention, attention weights and eviction
(oracle/serving.py): hand cases, library routines and invariants."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl


def test_prompt_attention_is_the_library_routine():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((40, 6, 8)), rng.standard_normal((40, 2, 8)), rng.standard_normal((40, 2, 8))
    offsets = [3, 3, 20, 21, 38]
    out, lse, spread, reach = oracle.prompt_attention_fp64(q, k, v, offsets)
    for a, b in zip(offsets, offsets[1:]):
        if a == b:
            continue
        t = [torch.from_numpy(x[a:b]).transpose(0, 1) for x in (q, np.repeat(k, 3, 1), np.repeat(v, 3, 1))]
        want = torch.nn.functional.scaled_dot_product_attention(*t, is_causal=True).transpose(0, 1).numpy()
        assert np.allclose(out[a:b], want, atol=1e-12)
        z = np.einsum("hd,hjd->hj", q[b - 1], t[1].numpy()) / np.sqrt(8)
        assert np.allclose(lse[b - 1], np.log(np.exp(z).sum(1)))
        assert (np.abs(out[a:b]) <= spread[a:b] + 1e-12).all() and (np.abs(z).max(1) <= reach[b - 1] + 1e-12).all()
    assert np.isnan(out[:3]).all() and np.isnan(out[38:]).all() and np.isnan(lse[38:]).all()


@pytest.mark.parametrize("rot", [None, (5, 9, 1 << 30, 77)])
def test_attention_weights_sum_to_the_group_size_and_give_the_output(rot):
    rng = np.random.default_rng(1)
    f = wl.CacheFormat(wl.INT8, wl.PER_TOKEN_HEAD)
    signs = None if rot is None else oracle.signs_from_words(rot, 64)
    oc = oracle.OracleCache(6, 16, 2, 64, f, f, signs)
    bits = lambda x: torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    x = rng.standard_normal((2, 60, 2, 64)).astype(np.float32)
    tables, ctx = np.array([[4, 0, 2], [5, -1, -1], [1, 3, -1]]), [45, 0, 20]
    slots = [tables[b][t // 16] * 16 + t % 16 for b in (0, 2) for t in range(ctx[b])][:60]
    oracle.quantize_write(oc, bits(x[0][:len(slots)]), bits(x[1][:len(slots)]), np.array(slots))
    ctx = [45, 0, len(slots) - 45]
    q = bits(rng.standard_normal((3, 6, 64)).astype(np.float32))
    w, reach = oracle.attention_weights_fp64(oc, q, tables, ctx, 50)
    assert np.allclose(w[[0, 2]].sum(-1), 3) and not w[1].any() and not w[0, :, 45:].any() and reach[1] == 0
    # one query head a kv head: the weights are the softmax that gives the output
    w, _ = oracle.attention_weights_fp64(oc, q[:, :2], tables, ctx, 50)
    t = np.arange(45)
    v = oracle.dequantize_cache_rows(oc, "v", tables[0][t // 16], t % 16)
    got = np.einsum("ht,thd->hd", w[0, :, :45], v)
    if rot is not None:
        got = oracle.unrotate_output_fp64(got, signs)
    assert np.allclose(got, oracle.paged_decode_fp64(oc, q[:, :2], tables, ctx)[0])


def test_eviction_hand_case():
    # one row of 7 tokens, one head: keep 4, the last one and the first one in any case
    codes = np.arange(2 * 16, dtype=np.uint8).reshape(2, 16, 1, 1)
    weights = np.array([[[0.0, 5, 1, 7, 7, 9, 0.5, 3]]], np.float32)
    tables = np.array([[1, -1]])
    kept = oracle.evict_tokens([4], [1], [1], [7], tables, [codes], weights)
    # kept: 0, 6, and of 1 .. 5 the two heaviest: 5 (9) and 3 (7, the lower of two); 3 -> 1 and 5 -> 2, 6 -> 3
    assert kept.tolist() == [4]
    assert codes[1, :8, 0, 0].tolist() == [16, 19, 21, 22, 20, 21, 22, 23] and codes[0, 3, 0, 0] == 3
    assert weights[0, 0].tolist() == [0, 7, 9, 0.5, 0, 0, 0, 3]


def test_eviction_keeps_what_it_should_whatever_the_sizes():
    rng = np.random.default_rng(4)
    for _ in range(150):
        n, length = int(rng.integers(0, 70)), 80
        k, w, p = (int(x) for x in rng.integers(0, 75, 3))
        ids = rng.permutation(9)[:5]
        tables = ids[None]
        codes = rng.permutation(9 * 16 * 2).reshape(9, 16, 2)
        weights = rng.integers(0, 6, (1, 2, length)).astype(np.float32)
        before, old = codes.copy(), weights.copy()
        kept = oracle.evict_tokens([k], [w], [p], [n], tables, [codes], weights)
        assert kept.tolist() == [min(n, k)]
        slot = lambda c, h, i: c[ids[i // 16], i % 16, h]  # noqa: E731
        if n <= k:
            assert (codes == before).all() and (weights == old).all()
            continue
        w = min(w, k)
        p = min(p, k - w)
        for h in range(2):
            now = [slot(codes, h, i) for i in range(k)]
            was = {slot(before, h, i): i for i in range(n)}
            held = [was[x] for x in now]
            assert len(set(held)) == k and held[:p] == list(range(p)) and held[k - w:] == list(range(n - w, n))
            lost = [old[0, h, i] for i in range(n) if i not in held]
            assert max(lost) <= min([old[0, h, i] for i in held[p:k - w]], default=9)
            assert [weights[0, h, i] for i in range(k)] == [old[0, h, i] for i in held]
            assert not weights[0, h, k:n].any() and (weights[0, h, n:] == old[0, h, n:]).all()
        untouched = [x for x in range(9) if x not in ids[:-(-k // 16)]]
        assert (codes[untouched] == before[untouched]).all()


def test_eviction_leaves_refused_rows_alone():
    codes = np.arange(4 * 16).reshape(4, 16, 1)
    weights = np.ones((5, 1, 32), np.float32)
    tables = np.array([[0, 7], [1, 2], [3, 3], [0, 1], [0, 1]])
    before, old = codes.copy(), weights.copy()
    refs = np.array([1, 2, 1, 1])
    kept = oracle.evict_tokens([5, 5, 5, -1, 5], [0] * 5, [0, 0, 0, 0, -2], [20, 30, 33, 9, 9], tables, [codes], weights, refs)
    assert kept.tolist() == [20, 30, 33, 9, 9] and (codes == before).all() and (weights == old).all()
