"""kvq_prompt_attention against the oracle's attention in float64."""
import math

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


def _draw(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


def check(q, k, v, offsets, out, lse, fill=None):
    """Rounding errors, element by element.  A score's D products are exact in
    FP32 (two BF16 factors); adding them, scaling and subtracting the maximum
    each round (or truncate: one step, 2^-23) at most what sum |q_i k_i| /
    sqrt(d) = `reach` bounds: D + 8 steps of it, and 4 of the logarithm's unit;
    the exponential adds 2^-21.  So a probability is off by a factor e^(2 zerr)
    (its own score and the sum's), and by 2^-8 as BF16 for the second product;
    its n terms, up to n rescalings among them, are added with n + 8 steps of
    sum p |v| = `spread`.  The output is rounded once, 2^-8."""
    as64 = lambda x: x.double().cpu().numpy()  # noqa: E731
    want, wlse, spread, reach = oracle.prompt_attention_fp64(as64(q), as64(k), as64(v), offsets)
    n, d = max(b - a for a, b in zip(offsets, offsets[1:])), q.shape[2]
    zerr = (d + 8) * 2.0 ** -23 * reach + 2.0 ** -21
    inside = ~np.isnan(wlse)
    got, glse = as64(out), as64(lse)
    p = np.expm1(2 * zerr)[..., None] + 2.0 ** -8 + (n + 8) * 2.0 ** -22
    moved = spread * p * (1 + p)
    bound = moved + 2.0 ** -8 * (np.abs(want) + moved) + 2.0 ** -126
    err = np.abs(got - want)[inside]
    assert np.isfinite(got[inside]).all()
    assert (err <= bound[inside]).all(), float((err / bound[inside]).max())
    lbound = zerr + (n + 8) * 2.0 ** -22 + 2.0 ** -22 * np.abs(wlse)
    lerr = np.abs(glse - wlse)[inside]
    assert (lerr <= lbound[inside]).all(), float((lerr / lbound[inside]).max())
    if fill is not None:                                     # rows outside every sequence: left as they were
        assert (got[~inside] == fill).all() and (glse[~inside] == fill).all()


def attend(q, k, v, offsets, fill=7.0, **kw):
    out = torch.full(q.shape, fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], fill, dtype=torch.float32, device="cuda")
    longest = max(b - a for a, b in zip(offsets, offsets[1:]))
    assert kvq.kvq_prompt_attention(q, k, v, _i32(offsets), longest, out=out, lse=lse, **kw) is out
    return out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (3, 1), (16, 4), (15, 3), (6, 1), (7, 1), (64, 8), (8, 8)])
def test_every_ratio_over_ragged_lengths(hq, hkv, d):
    gen = torch.Generator(device="cuda").manual_seed(hq * 100 + hkv * 10 + d)
    lens = [1, 0, 2, 130, 17, 0, 33, 257, 64, 127, 128, 129, 5]
    offsets = np.concatenate([[0], np.cumsum(lens)])
    n = int(offsets[-1])
    q, k, v = _draw(gen, n, hq, d), _draw(gen, n, hkv, d), _draw(gen, n, hkv, d)
    check(q, k, v, offsets, *attend(q, k, v, offsets), fill=7.0)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 384, 385,
                               511, 512, 513, 640, 1000])
def test_every_tile_edge(n):
    gen = torch.Generator(device="cuda").manual_seed(n)
    for hq, hkv, d in ((4, 1, 128), (2, 2, 64), (1, 1, 128)):
        q, k, v = _draw(gen, n + 3, hq, d), _draw(gen, n + 3, hkv, d), _draw(gen, n + 3, hkv, d)
        check(q, k, v, [2, n + 2], *attend(q, k, v, [2, n + 2]), fill=7.0)


def test_long_sequences():
    gen = torch.Generator(device="cuda").manual_seed(0)
    offsets = [0, 4097, 4098, 7201]
    q, k, v = _draw(gen, 7201, 8, 128), _draw(gen, 7201, 2, 128), _draw(gen, 7201, 2, 128)
    check(q, k, v, offsets, *attend(q, k, v, offsets))


def test_many_sequences():
    rng = np.random.default_rng(1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    offsets = np.concatenate([[0], np.cumsum(rng.integers(0, 40, 1500))])
    n = int(offsets[-1])
    q, k, v = _draw(gen, n, 2, 64), _draw(gen, n, 1, 64), _draw(gen, n, 1, 64)
    check(q, k, v, offsets, *attend(q, k, v, offsets))


def test_scores_of_hundreds_and_a_maximum_that_keeps_rising():
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = _draw(gen, 700, 4, 128), _draw(gen, 700, 1, 128), _draw(gen, 700, 1, 128)
    q[:, :] = 1.0
    k[:, :, 0] *= 20
    ramp = torch.linspace(-8, 8, 700, device="cuda")[:, None, None]
    for kk in (k * 20, (ramp + 0 * k).to(torch.bfloat16), (-ramp + 0 * k).to(torch.bfloat16)):
        check(q, kk, v, [0, 700], *attend(q, kk, v, [0, 700]))


def test_values_elsewhere_may_be_anything():
    """Rows behind the last sequence, gaps and other sequences hold infinities and NaN."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (_draw(gen, 900, h, 128) for h in (8, 2, 2))
    offsets = [10, 140, 141, 500, 777]
    clean = attend(q, k, v, offsets)
    for x in (q, k, v):
        x[:10], x[777:] = math.nan, math.inf
    dirty = attend(q, k, v, offsets)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])
    for x in (q, k, v):                                      # the first and the third sequence, too
        x[10:140], x[141:500] = -math.inf, math.nan
    dirty = attend(q, k, v, offsets)
    for a, b in ((140, 141), (500, 777)):
        assert torch.equal(clean[0][a:b], dirty[0][a:b]) and torch.equal(clean[1][a:b], dirty[1][a:b])


def test_parts_of_a_projection():
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = _draw(gen, 400, 20, 64)
    q, k, v = x.split((12, 4, 4), 1)
    offsets = [0, 150, 400]
    want = attend(q.contiguous(), k.contiguous(), v.contiguous(), offsets)
    got = attend(q, k, v, offsets)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    one = attend(q[7:8], k[7:8], v[7:8], [0, 1])
    assert torch.equal(one[0], v[7:8].repeat_interleave(3, 1))


def test_a_fresh_output_without_lse_and_a_side_stream():
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (_draw(gen, 300, h, 128) for h in (4, 2, 2))
    want, _ = attend(q, k, v, [0, 300])
    assert torch.equal(kvq.kvq_prompt_attention(q, k, v, _i32([0, 300]), 300), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        out = kvq.kvq_prompt_attention(q, k, v, _i32([0, 300]), 5000, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_captured_and_replayed_with_other_lengths():
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (_draw(gen, 600, h, 64) for h in (6, 2, 2))
    offsets, out, lse = _i32([0, 600, 600]), torch.zeros_like(q), torch.zeros(600, 6, device="cuda")
    ws = torch.empty(kvq.kvq_prompt_attention_workspace_size(2, 600, 6, 2), dtype=torch.uint8, device="cuda")
    call = lambda: kvq.kvq_prompt_attention(q, k, v, offsets, 600, out=out, lse=lse, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for o in ([0, 600, 600], [0, 1, 600], [5, 300, 555], [600, 600, 600]):
        offsets.copy_(_i32(o))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        check(q, k, v, o, out, lse, fill=7.0)


def test_two_calls_at_once():
    """Two streams, each with its own workspace, and two graphs that share one in turn."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = [[_draw(gen, 2500, h, 128) for h in (16, 4, 4)] for _ in range(2)]
    offsets = _i32([0, 1700, 2500])
    want = [kvq.kvq_prompt_attention(*y, offsets, 1700) for y in x]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(4):
        for k in range(2):
            got[k] = kvq.kvq_prompt_attention(*x[k], offsets, 1700, stream=streams[k])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ws = torch.empty(kvq.kvq_prompt_attention_workspace_size(2, 1700, 16, 4), dtype=torch.uint8, device="cuda")
    out, graphs = [torch.zeros_like(want[0]) for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for k in range(2):
        with torch.cuda.graph(graphs[k]):
            kvq.kvq_prompt_attention(*x[k], offsets, 1700, out=out[k], workspace=ws)
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_a_bound_far_above_the_lengths():
    gen = torch.Generator(device="cuda").manual_seed(10)
    q, k, v = (_draw(gen, 300, h, 64) for h in (8, 1, 1))
    want, _ = attend(q, k, v, [0, 1, 300])
    assert torch.equal(kvq.kvq_prompt_attention(q, k, v, _i32([0, 1, 300]), 1 << 24), want)


def test_bad_offsets_write_nothing():
    gen = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = (_draw(gen, 300, h, 64) for h in (2, 1, 1))
    def attempt(offsets, longest):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        kvq.kvq_prompt_attention(q, k, v, _i32(offsets), longest, out=out)
        return out, kvq.kvq_device_errors()
    for offsets in ([0, 200, 100], [-1, 100, 300], [0, 100, 301], [0, 2 ** 31 - 1, 100]):
        out, err = attempt(offsets, 300)
        assert err & kvq.DEVERR_GROUP_RANGE and bool((out == 7).all())
    out, err = attempt([0, 100, 300], 150)                   # one sequence longer than announced
    assert err == kvq.DEVERR_CONTEXT_RANGE and bool((out[100:] == 7).all())
    want, _ = attend(q, k, v, [0, 100])
    assert torch.equal(out[:100], want[:100])


def test_the_same_call_gives_the_same_bits():
    gen = torch.Generator(device="cuda").manual_seed(8)
    q, k, v = (_draw(gen, 3000, h, 128) for h in (8, 2, 2))
    offsets = [0, 900, 2999]
    first = attend(q, k, v, offsets)
    for _ in range(3):
        again = attend(q, k, v, offsets)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("d", [64, 128])
def test_a_sequence_gives_the_same_bits_in_any_batch(d):
    """Among thousands of units, which are taken ahead, and alone, where few are taken late."""
    lengths = [int(x) for x in np.random.default_rng(d).integers(1, 900, 60)] + [5000]
    offsets = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    gen = torch.Generator(device="cuda").manual_seed(d)
    q, k, v = (_draw(gen, offsets[-1], h, d) for h in (64, 8, 8))
    out, lse = attend(q, k, v, offsets)
    for s in [0, 7, 33, 59, 60]:
        a, b = offsets[s], offsets[s + 1]
        alone = attend(q[a:b], k[a:b], v[a:b], [0, b - a])
        assert torch.equal(alone[0], out[a:b]) and torch.equal(alone[1], lse[a:b])
