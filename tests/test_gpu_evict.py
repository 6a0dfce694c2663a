"""kvq_weigh_decode and kvq_evict_tokens against the oracle."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl

pytestmark = pytest.mark.gpu

kvq = None
TOK = wl.PER_TOKEN_HEAD
FMT = {"int8": wl.CacheFormat(wl.INT8, TOK), "fp8": wl.CacheFormat(wl.FP8, TOK), "int4": wl.CacheFormat(wl.INT4, TOK),
       "v4": wl.CacheFormat(wl.INT4, wl.PER_TOKEN_GROUP, 32), "v2": wl.CacheFormat(wl.INT2, wl.PER_TOKEN_GROUP, 32)}


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


def _bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def make(k, v, h, d, ctx, seed=0, rot=None, spare=3, scale=1.0):
    """A cache of rows of the given contexts in blocks of any order, here and in the oracle."""
    rng = np.random.default_rng(seed)
    held = [-(-n // 16) for n in ctx]
    nb = sum(held) + spare
    ids, at = rng.permutation(nb), 0
    tables = np.full((len(ctx), max(held) + 1), -1)
    for r, x in enumerate(held):
        tables[r, :x] = ids[at:at + x]
        at += x
    fmt = kvq.cache_format(FMT[k], FMT[v], h, d, nb, rotation_signs=rot)
    cache = kvq.allocate_cache(fmt)
    oc = oracle.OracleCache(nb, 16, h, d, FMT[k], FMT[v], None if rot is None else oracle.signs_from_words(rot, d))
    slots = np.concatenate([tables[r][np.arange(n) // 16] * 16 + np.arange(n) % 16 for r, n in enumerate(ctx)]).astype(np.int64)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((2, len(slots), h, d), generator=gen, device="cuda") * scale).to(torch.bfloat16)
    kvq.kvq_quantize_write(x[0], x[1], torch.from_numpy(slots).cuda(), fmt, cache)
    for w in ("k", "v"):
        oc.codes[w][...] = cache[w + "_cache"].cpu().numpy()
        oc.scales[w][...] = cache[w + "_scale"].cpu().numpy()
    return fmt, cache, oc, tables, gen


def check_weights(got, before, oc, q, tables, ctx, fmt):
    """A score's D products (exact codes, BF16 or two-part f16 queries) add up in
    FP32 with a step (2^-23) each of at most reach = the largest sum |q_i k_i| /
    sqrt(d); its scale, the maximum and the query's second part a few more.  The
    weight is off by the factor e^(2 zerr), 2^-21 of the exponential and n steps
    of the sum; G of them and the entry before are added with a step each."""
    length = got.shape[2]
    want, reach = oracle.attention_weights_fp64(oc, _bits(q), tables, ctx, length)
    g = q.shape[1] // fmt.num_kv_heads
    n = np.array(ctx)[:, None, None]
    zerr = ((fmt.head_dim + 16) * 2.0 ** -23 * reach + 2.0 ** -20)[:, None, None]
    bound = want * (np.expm1(2 * zerr) + n * 2.0 ** -23) + (g + 1) * 2.0 ** -23 * (want + np.abs(before))
    err = np.abs(got.double().cpu().numpy() - (before + want))
    assert (err <= bound + 2.0 ** -126).all(), float((err / (bound + 2.0 ** -126)).max())
    outside = np.broadcast_to(np.arange(length) >= n, want.shape)
    assert (got.cpu().numpy()[outside] == before[outside].astype(np.float32)).all()


@pytest.mark.parametrize("k,v,h,g,d,rot", [
    ("int8", "int8", 2, 2, 64, None), ("fp8", "fp8", 8, 4, 128, None), ("int8", "v4", 8, 8, 128, None),
    ("int4", "v4", 8, 4, 128, (1, 2, 3, 4)), ("fp8", "v2", 3, 5, 128, None), ("int4", "int8", 1, 1, 64, None),
    ("int8", "fp8", 7, 7, 128, (9, 8, 7, 6)), ("fp8", "v4", 5, 3, 64, None)])
def test_weights_and_the_same_output(k, v, h, g, d, rot):
    ctx = [0, 1, 15, 16, 17, 300, 33, 1000, 0]
    fmt, cache, oc, tables, gen = make(k, v, h, d, ctx, seed=h * 10 + g, rot=rot)
    q = torch.randn((len(ctx), h * g, d), generator=gen, device="cuda").to(torch.bfloat16)
    for length in (1000, 1024, 1013):                        # entries of a row need not be aligned
        weights = torch.rand((len(ctx), h, length), generator=gen, device="cuda")
        before = weights.double().cpu().numpy()
        out = kvq.kvq_weigh_decode(q, fmt, cache, _i32(tables), _i32(ctx), 1000, weights)
        assert torch.equal(out, kvq.kvq_paged_decode(q, fmt, cache, _i32(tables), _i32(ctx), 1000))
        check_weights(weights, before, oc, q, tables, ctx, fmt)


def test_large_scores_and_many_short_rows():
    ctx = [int(x) for x in np.random.default_rng(0).integers(0, 50, 300)]
    fmt, cache, oc, tables, gen = make("int8", "int8", 2, 64, ctx, seed=1, scale=6.0)
    q = (torch.randn((len(ctx), 4, 64), generator=gen, device="cuda") * 5).to(torch.bfloat16)
    weights = torch.zeros((len(ctx), 2, 64), device="cuda")
    kvq.kvq_weigh_decode(q, fmt, cache, _i32(tables), _i32(ctx), 64, weights)
    check_weights(weights, np.zeros(weights.shape), oc, q, tables, ctx, fmt)


def test_weights_of_what_the_decode_leaves_out():
    ctx = [40, 100, 60]
    fmt, cache, oc, tables, gen = make("fp8", "fp8", 2, 128, ctx, seed=2)
    q = torch.randn((3, 8, 128), generator=gen, device="cuda").to(torch.bfloat16)
    weights = torch.zeros((3, 2, 128), device="cuda")
    out = kvq.kvq_weigh_decode(q, fmt, cache, _i32(tables), _i32([40, -3, 60]), 128, weights)
    assert kvq.kvq_device_errors() == kvq.DEVERR_CONTEXT_RANGE and not weights[1].any() and not out[1].any()
    check_weights(weights, np.zeros(weights.shape), oc, q, tables, [40, 0, 60], fmt)
    broken = tables.copy()
    broken[1, 2] = 10 ** 6
    weights.zero_()
    kvq.kvq_weigh_decode(q, fmt, cache, _i32(broken), _i32(ctx), 128, weights)
    assert kvq.kvq_device_errors() == kvq.DEVERR_BLOCK_RANGE
    assert not weights[1, :, 32:48].any() and bool((weights[1, :, :32] > 0).all()) and bool((weights[1, :, 48:100] > 0).all())


def test_weights_captured_replayed_and_on_a_side_stream():
    ctx = [70, 5, 200]
    fmt, cache, oc, tables, gen = make("int8", "v4", 4, 128, ctx, seed=3)
    q = torch.randn((3, 16, 128), generator=gen, device="cuda").to(torch.bfloat16)
    t, c = _i32(tables), _i32(ctx)
    once = torch.zeros((3, 4, 256), device="cuda")
    want = kvq.kvq_weigh_decode(q, fmt, cache, t, c, 256, once)
    ws = torch.empty(kvq.kvq_weigh_decode_workspace_size(fmt, 3, 16, 256), dtype=torch.uint8, device="cuda")
    weights, out = torch.zeros_like(once), torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_weigh_decode(q, fmt, cache, t, c, 256, weights, out=out, workspace=ws)
    for k in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(weights, once + once + once)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    weights.zero_()
    torch.cuda.synchronize()
    got = kvq.kvq_weigh_decode(q, fmt, cache, t, c, 256, weights, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(weights, once)


def test_weights_of_two_calls_at_once():
    """Two streams, each with its own workspace."""
    ctx = [900, 30, 1200]
    fmt, cache, oc, tables, gen = make("fp8", "v4", 8, 128, ctx, seed=8)
    t, c = _i32(tables), _i32(ctx)
    q = torch.randn((2, 3, 32, 128), generator=gen, device="cuda").to(torch.bfloat16)
    weights = torch.zeros((2, 3, 8, 1200), device="cuda")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = [None, None]
    for _ in range(5):
        for k in range(2):
            out[k] = kvq.kvq_weigh_decode(q[k], fmt, cache, t, c, 1200, weights[k], stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        once = torch.zeros((3, 8, 1200), device="cuda")
        assert torch.equal(kvq.kvq_weigh_decode(q[k], fmt, cache, t, c, 1200, once), out[k])
        five = torch.zeros_like(once)
        for _ in range(5):
            five += once
        assert torch.equal(five, weights[k])


def test_weights_of_eight_thousand_rows():
    rng = np.random.default_rng(3)
    ctx = [int(x) for x in rng.integers(0, 20, 8192) * (rng.random(8192) < 0.3)]
    fmt, cache, oc, tables, gen = make("int8", "int8", 1, 64, ctx, seed=9)
    q = torch.randn((len(ctx), 3, 64), generator=gen, device="cuda").to(torch.bfloat16)
    weights = torch.zeros((len(ctx), 1, 20), device="cuda")
    kvq.kvq_weigh_decode(q, fmt, cache, _i32(tables), _i32(ctx), 20, weights)
    some = sorted(set(rng.integers(0, 8192, 300).tolist()) | {0, 8191})
    check_weights(weights[some], np.zeros((len(some), 1, 20)), oc, q[some], tables[some], [ctx[i] for i in some], fmt)


class Both:
    """The same cache and weights on the device and in the oracle."""

    def __init__(self, k, v, h, d, ctx, seed, length=None, weights=None, rot=None):
        self.fmt, self.cache, self.oc, self.tables, self.gen = make(k, v, h, d, ctx, seed=seed, rot=rot)
        self.ctx = list(ctx)
        length = length or max(ctx)
        rng = np.random.default_rng(seed)
        self.w = (rng.random((len(ctx), h, length)) ** 7).astype(np.float32) if weights is None else weights
        self.arrays = [self.oc.codes["k"], self.oc.codes["v"], self.oc.scales["k"], self.oc.scales["v"]]
        self.dw, self.dt, self.dc = torch.from_numpy(self.w).cuda(), _i32(self.tables), _i32(ctx)

    def evict(self, keep, recent, pinned=None, refs=None, **kw):
        want = oracle.evict_tokens(keep, recent, [0] * len(keep) if pinned is None else pinned, self.ctx, self.tables,
                                   self.arrays, self.w, refs)
        pool = None if refs is None else dict(ref_counts=_i32(refs))
        got = kvq.kvq_evict_tokens(_i32(keep), self.dc, self.dt, self.fmt, self.cache, self.dw, _i32(recent),
                                   pinned_lens=None if pinned is None else _i32(pinned), pool=pool, **kw)
        torch.cuda.synchronize()
        assert np.array_equal(got.cpu().numpy(), want)
        self.check()
        return want

    def check(self):
        assert np.array_equal(self.dw.cpu().numpy(), self.w, equal_nan=True)
        for name, x in zip(("k_cache", "v_cache", "k_scale", "v_scale"), self.arrays):
            assert np.array_equal(self.cache[name].cpu().numpy(), x), name


@pytest.mark.parametrize("k,v,h,d", [("int8", "int8", 2, 64), ("fp8", "fp8", 8, 128), ("int4", "v4", 4, 128),
                                     ("int8", "v2", 3, 128), ("int4", "v4", 5, 64), ("fp8", "v4", 7, 64)])
def test_formats_and_lengths(k, v, h, d):
    ctx = [0, 1, 2, 16, 17, 100, 333, 700, 64, 65]
    s = Both(k, v, h, d, ctx, seed=h, length=701)
    s.evict([0, 0, 1, 9, 16, 100, 50, 650, 1, 64], [0, 0, 0, 3, 16, 5, 60, 40, 0, 1], [0, 1, 5, 0, 3, 0, 7, 4, 1, 70])
    s.evict([0] * 10, [4] * 10)                              # everything goes


@pytest.mark.parametrize("n,k,w,p", [
    (40, 39, 38, 0), (40, 39, 0, 39), (40, 39, 39, 39), (5000, 4999, 1024, 1), (5000, 4999, 4998, 0), (5000, 2500, 0, 0),
    (5000, 33, 1, 1), (5000, 1, 1, 1), (5000, 1, 0, 0), (5000, 4000, 3900, 50), (2100, 2048, 1030, 16), (4097, 4096, 0, 0),
    (9000, 4500, 100, 4), (40, 20, 2 ** 31 - 1, 2 ** 31 - 1), (40, 20, 0, 2 ** 31 - 1)])
def test_windows_that_overlap_and_lists_that_are_full(n, k, w, p):
    Both("int8", "int8", 2, 64, [n], seed=k + w).evict([k], [w], [p])


def test_all_heavy_ones_last_and_all_first():
    up = np.broadcast_to(np.arange(1000, dtype=np.float32), (1, 2, 1000)).copy()
    Both("int8", "int8", 2, 64, [1000], seed=1, weights=up).evict([500], [0])     # every kept token moves
    Both("int8", "int8", 2, 64, [1000], seed=1, weights=-up).evict([500], [0])    # none does


@pytest.mark.parametrize("kind", ["zero", "few", "subnormal", "special", "negative", "huge"])
def test_ties_and_odd_weights(kind):
    rng = np.random.default_rng(5)
    w = np.zeros((2, 3, 3001), np.float32)
    if kind == "few":
        w = rng.integers(0, 3, w.shape).astype(np.float32)
    elif kind == "subnormal":
        w = (rng.integers(0, 50, w.shape) * 2.0 ** -149).astype(np.float32)
    elif kind == "special":
        w = rng.choice(np.array([0.0, -0.0, 1.0, np.inf, -np.inf, np.nan, -np.nan, 3.4e38], np.float32), w.shape)
    elif kind == "negative":
        w = rng.standard_normal(w.shape).astype(np.float32)
    elif kind == "huge":
        w = (1e38 * rng.random(w.shape)).astype(np.float32)
    Both("int8", "int8", 3, 64, [3001, 2990], seed=2, weights=w).evict([1500, 2900], [10, 200], [3, 0])


@pytest.mark.parametrize("h,rows,length,kind", [(1, 1, 20000, "few"), (2, 3, 9001, "zero"), (4, 9, 8192, "rand"), (1, 70, 8192, "few"),
                                                (8, 40, 8195, "few"), (2, 1, 33000, "rand"), (3, 1, 70001, "few"), (1, 1, 140003, "few"),
                                                (7, 30, 16390, "few")])
def test_long_rows_with_ties(h, rows, length, kind):
    """One CTA, a cluster of two, four and eight for each (row, head); the longest one's keys are not held."""
    rng = np.random.default_rng(length)
    w = np.zeros((rows, h, length), np.float32) if kind == "zero" else rng.integers(0, 4, (rows, h, length)).astype(np.float32)
    if kind == "rand":
        w = rng.random(w.shape).astype(np.float32) ** 5
    ctx = [length] + [int(x) for x in rng.integers(0, 150, rows - 1)]
    if rows < 10:
        ctx[-1] = length - 77
    keep = [length // 2 if n > 1000 else n // 2 for n in ctx]
    s = Both("int8", "int8", h, 64, ctx, seed=7, weights=w)
    s.evict(keep, [int(x) for x in rng.integers(0, 70, rows)], [int(x) for x in rng.integers(0, 40, rows)])
    s.ctx = keep
    s.dc = _i32(keep)
    s.evict([max(0, n - 3) for n in keep], [1] * rows)


def test_rows_that_are_refused_stay_as_they_are():
    s = Both("fp8", "v4", 2, 128, [100, 100, 100, 100, 100, 100], seed=3, length=112)
    refs = np.ones(s.fmt.num_blocks, np.int64)
    refs[s.tables[0, 1]] = 2                                 # a block of row 0 that another row holds
    refs[s.tables[1, 6]] = 2                                 # of row 1, past what is kept: only read
    refs[s.tables[2, 0]] = 3                                 # of row 2, within what is pinned
    s.tables[3, 5] = s.fmt.num_blocks
    s.dt = _i32(s.tables)
    kept = s.evict([50, 50, 50, 50, -1, 50], [4] * 5 + [-4], [0, 0, 16, 0, 0, 0], refs=refs)
    assert kept.tolist() == [100, 50, 50, 100, 100, 100]
    assert kvq.kvq_device_errors() == kvq.DEVERR_POOL_STATE | kvq.DEVERR_BLOCK_RANGE | kvq.DEVERR_CONTEXT_RANGE
    s.ctx[0], s.dc[0] = 113, 113                             # longer than the weights
    assert s.evict([50] * 6, [4] * 6)[0] == 113
    assert kvq.kvq_device_errors() == kvq.DEVERR_BLOCK_RANGE | kvq.DEVERR_CONTEXT_RANGE


def test_many_rows():
    rng = np.random.default_rng(6)
    ctx = [int(x) for x in rng.integers(0, 90, 700)]
    s = Both("int8", "int8", 8, 64, ctx, seed=4, length=96)
    s.evict(rng.integers(0, 90, 700).tolist(), rng.integers(0, 30, 700).tolist(), rng.integers(0, 9, 700).tolist())


def test_captured_and_replayed_as_the_weights_change():
    s = Both("int8", "v4", 4, 128, [500, 90], seed=5)
    keep, recent, pinned = _i32([400, 64]), _i32([32, 8]), _i32([4, 0])
    kept = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(kvq.kvq_evict_workspace_size(2, 4, 500), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_evict_tokens(keep, s.dc, s.dt, s.fmt, s.cache, s.dw, recent, pinned_lens=pinned, kept_lens=kept, workspace=ws)
    for k in range(3):
        w = (np.random.default_rng(k).random(s.w.shape) ** 5).astype(np.float32)
        s.w[...] = w
        s.dw.copy_(torch.from_numpy(w))
        oracle.evict_tokens([400, 64], [32, 8], [4, 0], s.ctx, s.tables, s.arrays, s.w)
        graph.replay()
        torch.cuda.synchronize()
        s.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.evict([300, 60], [5, 5], stream=side)


def test_a_budget_held_over_many_steps():
    """Prompts, decode steps whose weights add up, evictions and releases, as a
    server runs them; the decode after every eviction is the attention over what
    is kept."""
    h, g, d, rows, budget = 2, 4, 128, 3, 96
    f = FMT["fp8"]
    nb, width = 60, 16
    fmt = kvq.cache_format(f, f, h, d, nb)
    cache, pool = kvq.allocate_cache(fmt), kvq.allocate_pool(nb)
    oc = oracle.OracleCache(nb, 16, h, d, f, f)
    gen = torch.Generator(device="cuda").manual_seed(9)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    ctx, tables = _i32([0] * rows), torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    weights = torch.zeros((rows, h, width * 16), device="cuda")
    n = [150, 20, 200]
    offsets, slots, _ = kvq.kvq_assign_blocks(_i32(n), ctx, tables, pool, sum(n) + 7)
    q, k, v = draw(sum(n) + 7, h * g, d), draw(sum(n) + 7, h, d), draw(sum(n) + 7, h, d)
    out = kvq.kvq_prompt_attention(q, k, v, offsets, 200)    # the offsets of the assignment are the prompts'
    kvq.kvq_quantize_write(k, v, slots, fmt, cache)
    # the last token of a prompt has no later ones: nearly the decode's attention (over FP8 codes)
    last = (offsets[1:] - 1).long()
    near = kvq.kvq_paged_decode(q[last], fmt, cache, tables, ctx, width * 16)
    assert float((out[last].float() - near).abs().max()) < 0.1
    for step in range(40):
        _, slots, _ = kvq.kvq_assign_blocks(_i32([1] * rows), ctx, tables, pool, rows)
        kvq.kvq_quantize_write(draw(rows, h, d), draw(rows, h, d), slots, fmt, cache)
        q = draw(rows, h * g, d)
        before = weights.double().cpu().numpy()
        out = kvq.kvq_weigh_decode(q, fmt, cache, tables, ctx, width * 16, weights)
        for w in ("k", "v"):
            oc.codes[w][...], oc.scales[w][...] = cache[w + "_cache"].cpu().numpy(), cache[w + "_scale"].cpu().numpy()
        t, c = tables.cpu().numpy(), ctx.tolist()
        assert np.abs(out.double().cpu().numpy() - oracle.paged_decode_fp64(oc, _bits(q), t, c)).max() < 2e-3
        check_weights(weights, before, oc, q, t, c, fmt)
        if step % 8 == 7:
            w = weights.cpu().numpy()
            arrays = [oc.codes["k"], oc.codes["v"], oc.scales["k"], oc.scales["v"]]
            want = oracle.evict_tokens([budget] * rows, [16] * rows, [4] * rows, c, t, arrays, w, pool["ref_counts"].cpu().numpy())
            kept = kvq.kvq_evict_tokens(_i32([budget] * rows), ctx, tables, fmt, cache, weights, _i32([16] * rows),
                                        pinned_lens=_i32([4] * rows), pool=pool)
            kvq.kvq_release_blocks(kept, ctx, tables, pool)
            assert kept.tolist() == want.tolist() == ctx.tolist() and max(want) <= budget
            assert np.array_equal(weights.cpu().numpy(), w)
            for name, x in zip(("k_cache", "v_cache", "k_scale", "v_scale"), arrays):
                assert np.array_equal(cache[name].cpu().numpy(), x), name
    assert int(pool["free_count"]) == nb - sum(-(-x // 16) for x in ctx.tolist())


def test_no_rows_and_no_positions():
    fmt, cache, oc, tables, gen = make("int8", "int8", 2, 64, [20, 5], seed=4)
    q = torch.randn((2, 4, 64), generator=gen, device="cuda").to(torch.bfloat16)
    none = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    assert kvq.kvq_weigh_decode(q[:0], fmt, cache, _i32(tables)[:0], _i32([]), 20, none(0, 2, 20)).shape == (0, 4, 64)
    assert not kvq.kvq_weigh_decode(q, fmt, cache, _i32(tables), _i32([0, 0]), 0, none(2, 2, 0)).any()
    args = (_i32(tables), fmt, cache)
    assert kvq.kvq_evict_tokens(_i32([]), _i32([]), args[0][:0], fmt, cache, none(0, 2, 20), _i32([])).shape == (0,)
    assert kvq.kvq_evict_tokens(_i32([3, 0]), _i32([0, 0]), *args, none(2, 2, 0), _i32([1, 1])).tolist() == [0, 0]
    assert kvq.kvq_device_errors() == 0
    assert kvq.kvq_evict_tokens(_i32([3, 0]), _i32([0, 5]), *args, none(2, 2, 0), _i32([1, 1])).tolist() == [0, 5]
    assert kvq.kvq_device_errors() == kvq.DEVERR_CONTEXT_RANGE


@pytest.mark.parametrize("rows,h,g,d", [(1, 8, 4, 128), (32, 8, 4, 128), (33, 8, 4, 128), (64, 8, 2, 64), (65, 8, 2, 64), (1, 1, 1, 64)])
def test_few_and_many_rows_to_merge(rows, h, g, d):
    """On either side of the rows that one warp each merges."""
    rng = np.random.default_rng(rows)
    ctx = [2500] + [int(x) for x in rng.integers(0, 200, rows - 1)]
    fmt, cache, oc, tables, gen = make("fp8", "fp8", h, d, ctx, seed=rows)
    q = torch.randn((rows, h * g, d), generator=gen, device="cuda").to(torch.bfloat16)
    weights = torch.zeros((rows, h, 2500), device="cuda")
    out = kvq.kvq_weigh_decode(q, fmt, cache, _i32(tables), _i32(ctx), 2500, weights)
    assert torch.equal(out, kvq.kvq_paged_decode(q, fmt, cache, _i32(tables), _i32(ctx), 2500))
    ref = oracle.paged_decode_fp64(oc, _bits(q), tables, np.array(ctx))
    err = np.abs(out.double().cpu().numpy() - ref)
    assert err.max() <= 2e-3 and (err <= 1e-2 * np.abs(ref))[np.abs(ref) >= 0.2].all()   # the decode's own bounds
    check_weights(weights, np.zeros(weights.shape), oc, q, tables, ctx, fmt)


@pytest.mark.parametrize("h,rows,length", [(8, 60, 8190), (8, 60, 4097), (8, 50, 4097), (2, 3, 4096), (1, 500, 8192), (1, 2, 40000), (2, 1, 16385)])
def test_long_rows_among_few_and_many(h, rows, length):
    """Either number of threads, on both sides of their bounds."""
    rng = np.random.default_rng(length + rows)
    w = (rng.random((rows, h, length)) ** 5).astype(np.float32)
    w[:, :, ::7] = 0.25
    ctx = [length] + [int(x) for x in rng.integers(0, 40, rows - 1)]
    keep = [n // 3 for n in ctx]
    Both("int8", "int8", h, 64, ctx, seed=8, weights=w).evict(keep, [n // 5 for n in keep], [n // 9 for n in keep])


@pytest.mark.parametrize("h,rows,length", [(8, 18, 20001), (8, 18, 32768), (8, 8, 40003), (8, 8, 65536), (8, 4, 70002)])
def test_long_rows_that_share_the_sms(h, rows, length):
    """Selections by CTAs of 1024 threads, one and clusters of two and four."""
    rng = np.random.default_rng(length)
    w = rng.integers(0, 50, (rows, h, length)).astype(np.float32)
    ctx = [int(x) for x in rng.integers(0, 60, rows)]
    ctx[rows // 2] = length - 1
    keep = [n // 2 for n in ctx]
    Both("int8", "int8", h, 64, ctx, seed=9, weights=w, length=length).evict(keep, [n // 6 for n in keep], [n // 8 for n in keep])
