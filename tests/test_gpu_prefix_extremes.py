"""kvq_prefix_decode on long prefixes and at the ends of its operands' ranges, against
float64 attention under the softmax-weighted bound of tests/_prefix_bound.py, which
sees a lost tile."""
import numpy as np
import pytest
import torch

import oracle
from tests import _helpers as H
from tests import _prefix_bound as bound
from tests import test_gpu_prefix_decode as base

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


def rows_of(s, b, h):
    """q [d], k and v [n, d] of one row in float64, in the cache's basis."""
    n = int(s.ctx[b])
    t = np.arange(n)
    kv = h // (s.hq // s.hkv)
    k, v = (oracle.dequantize_cache_rows(s.oc, w, s.table[b][t // 16], t % 16)[:, kv] for w in "kv")
    q = oracle.bf16_bits_to_f32(H.bits(s.q[b])).astype(np.float64)
    if s.oc.rotation is not None:
        q = oracle.rotate_query_fp64(q, s.oc.rotation)
    return q[h], k, v


def check(s, out, skip=()):
    """Every row but those in `skip` inside its bound."""
    got = out.float().cpu().numpy().astype(np.float64)
    worst = 0.0
    for b in range(len(s.ctx)):
        for h in range(s.hq):
            if (b, h) in skip:
                continue
            if s.ctx[b] == 0:
                assert (got[b, h] == 0).all()
                continue
            o, err = bound.row_bound(*rows_of(s, b, h), roundings=int(s.fmt.k_gran == "block_channel" or s.oc.rotation is not None))
            if s.oc.rotation is not None:
                o, err = oracle.unrotate_output_fp64(o[None], s.oc.rotation)[0], np.full_like(err, err.sum() / s.d)
            miss = np.abs(got[b, h] - o) / bound.rounded(o, err)
            assert np.isfinite(got[b, h]).all() and miss.max() <= 1.0, (b, h, miss.max())
            worst = max(worst, float(miss.max()))
    print(f"[prefix] error / weighted bound {worst:.3f}")


@pytest.mark.parametrize("k,v,hq,hkv,prefix,n,rot", [
    ("fp8", "fp8", 8, 2, 5003, 3, False), ("int8", "int8", 4, 1, 5003, 40, False), ("int8c", "int4g", 16, 2, 4999, 4, False),
    ("int2c", "int2g", 8, 1, 4100, 3, False), ("int4", "int4g", 8, 1, 3001, 3, True), ("fp8", "int4g", 8, 1, 2900, 40, False),
    ("int8", "fp8", 6, 3, 500, 5, False)])
def test_long_prefixes_under_the_weighted_bound(k, v, hq, hkv, prefix, n, rot):
    s = base.Batch(k, v, hq=hq, hkv=hkv, groups=[(prefix, [prefix + 3 * i for i in range(n)])], rot=rot, seed=31,
                   outliers=False)
    check(s, s.run())


@pytest.mark.parametrize("k,v,d,rows", [("fp8", "fp8", 128, 20), ("int8", "int8", 128, 40), ("int4", "int4g", 128, 20),
                                        ("int8", "fp8", 64, 40), ("fp8", "int4g", 64, 20), ("int4", "int8", 64, 20)])
def test_per_token_k_codes_are_exact_under_outliers(k, v, d, rows):
    """Scores of hundreds, from outlier channels and tokens: a rounding of K would
    move them by tenths."""
    s = base.Batch(k, v, hq=16, hkv=2, d=d, groups=[(600, [600 + 5 * i for i in range(rows)])], seed=36)
    s.q *= 4
    check(s, s.run())


@pytest.mark.parametrize("k", ["int8", "fp8", "int4", "int8c"])
@pytest.mark.parametrize("down", [30, 41, 50, 100])
def test_tiny_queries_against_tiny_scales(k, down):
    """Scores that vanish beside masked positions (the prefix ends inside a
    tile): the mean of V, no NaN."""
    s = base.Batch(k, "int8", groups=[(200, [201, 230, 150, 210, 199])], seed=32)
    s.cache["k_scale"] *= 2.0 ** -down
    s.oc.scales["k"] = s.cache["k_scale"].cpu().numpy()
    s.q[0] = 0
    s.q[1] *= 2.0 ** -90
    s.q[2] *= 2.0 ** -60
    s.q[3] *= 2.0 ** down                               # (scores of the usual size)
    s.q[4, ::2] = 0
    check(s, s.run())


def test_non_finite_queries_stay_in_their_rows():
    """A row that holds NaN or infinity comes back NaN, also where it ends inside
    the prefix; the others are as they should be, and a padded row is 0 whatever it holds."""
    s = base.Batch("fp8", "int8", groups=[(200, [150, 201, 0, 230, 333])], seed=33)
    s.q[0, 1, 5] = float("nan")
    s.q[1, 0] = float("nan")
    s.q[2] = float("nan")
    s.q[3, 2, 0] = float("inf")
    s.q[4, 7, 127] = float("-inf")
    out = s.run()
    bad = [(0, 1), (1, 0), (3, 2), (4, 7)]
    assert all(torch.isnan(out[b, h]).all() for b, h in bad)
    check(s, out, skip=bad)


def test_the_longest_context():
    """2^31 - 16 positions, all in one block: its 16 tokens' softmax.  FP32 sums of
    2^31 terms: a stream of a CTA (one of 304) adds 2^24 / 304 tiles, eight times
    each, every addition off by up to 2^-23 of what it has: 441505 2^-23 = 0.053 of A
    for the outputs, an eighth of it for l."""
    width, d = 2 ** 27 - 1, 64
    fmt = kvq.cache_format(base.INT8, base.INT8, 1, d, 1)
    cache = kvq.allocate_cache(fmt)
    gen = torch.Generator(device="cuda").manual_seed(35)
    x = torch.randn((2, 16, 1, d), generator=gen, device="cuda").to(torch.bfloat16)
    q = torch.randn((2, 2, d), generator=gen, device="cuda").to(torch.bfloat16)
    kvq.kvq_quantize_write(x[0], x[1], torch.arange(16, device="cuda"), fmt, cache)
    table = torch.zeros((2, width), dtype=torch.int32, device="cuda")
    n = 16 * width
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device="cuda")  # noqa: E731
    out = kvq.kvq_prefix_decode(q, fmt, cache, table, i32([n, n]), n, i32([0, 2]), i32([2 ** 31 - 1]), 2 ** 31 - 1)
    torch.cuda.synchronize()
    k, v = ((cache[w + "_cache"].view(torch.int8).double() * cache[w + "_scale"].double()[..., None])[0, :, 0]
            for w in "kv")
    p = torch.softmax(q.double() @ k.t() / d ** 0.5, -1)
    want, a = p @ v, p @ v.abs()
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (0.053 * 9 / 8 + 2.0 ** -9) * a).all()


def test_the_default_stream_given_by_its_handle(monkeypatch):
    """Handle 0 is the default stream: what the call makes is allocated there."""
    s = base.Batch(groups=[(300, [310, 320, 333])], seed=34)
    want, args = s.run(), s.args()
    plain, where = torch.empty, []

    def empty(*a, **k):
        where.append(torch.cuda.current_stream().cuda_stream)
        return plain(*a, **k)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", empty)
    with torch.cuda.stream(side):
        out = kvq.kvq_prefix_decode(*args, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and where == [0, 0]
