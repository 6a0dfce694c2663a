"""kvq_prompt_attention over thousands of keys, where every row's bound goes by
its own number of keys: a mask that is off by one key shows."""
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


def attend(q, k, v, offsets):
    out = torch.full(q.shape, math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], math.nan, device="cuda")
    kvq.kvq_prompt_attention(q, k, v, torch.tensor(offsets, dtype=torch.int32, device="cuda"), max(np.diff(offsets)), out=out, lse=lse)
    as64 = lambda x: x.double().cpu().numpy()  # noqa: E731
    return as64(out), as64(lse), oracle.prompt_attention_fp64(as64(q), as64(k), as64(v), offsets)


def sum_steps(offsets):
    """Steps of 2^-24 that a row's sum of exponentials is off by at most: its keys are
    added in four chains of 32 a tile of 128 and two more additions, each tile's sum
    once (34 + tiles); a tile may raise the reference, which multiplies what was there
    by an exponential (its own error 2^-22, four steps, that of its argument counted
    with the scores, and one for the product: 5 tiles)."""
    n = np.concatenate([np.arange(1, b - a + 1) for a, b in zip(offsets, offsets[1:])])
    tiles = -(-n // 128)
    return 34 + 6 * tiles


def score_error(reach, d):
    """D products, exact in FP32, are added, scaled and shifted with a step (2^-23,
    truncation included) each of at most sum |q_i k_i| / sqrt(d); the exponential
    adds 2^-21."""
    return (d + 8) * 2.0 ** -23 * reach + 2.0 ** -21


def check_lse(got, want, reach, d, offsets):
    """The scores' errors, the sum's, and the logarithm's: of a sum below 2^6 times the
    keys, so below 32, a step of 2^-19, then added to the reference and multiplied."""
    bound = score_error(reach, d) + (sum_steps(offsets) * 2.0 ** -24)[:, None] + 2.0 ** -19 + 2.0 ** -21 * np.abs(want)
    err = np.abs(got - want)
    assert (err <= bound).all(), float((err / bound).max())
    return bound


def check_out(got, want, spread, reach, d, offsets):
    """p is off by its score's and the sum's error, and by 2^-8 as BF16; the second
    product's terms are added, and rescaled with the sum, with a step of sum p |v| for
    each of its 8 instructions a tile of 16 terms (24 steps with the terms' own) and
    each raise (6); the output is rounded once, 2^-8."""
    tiles = (sum_steps(offsets) - 34)[:, None] / 6
    p = np.expm1(2 * score_error(reach, d)) + 2.0 ** -8 + (8 * 24 + 6) * tiles * 2.0 ** -23 + (34 + 6 * tiles) * 2.0 ** -24
    moved = spread * (p * (1 + p))[..., None]
    bound = moved + 2.0 ** -8 * (np.abs(want) + moved) + 2.0 ** -126
    err = np.abs(got - want)
    assert (err <= bound).all(), float((err / bound).max())


# few units of many tiles (taken late) and units that are taken ahead; 128 / 3, 128 / 5
# and 128 / 7 rows of a tile are no whole number
SHAPES = [(64, 3, 1, [0, 5003]), (64, 1, 1, [0, 4097, 4098, 6500]), (64, 14, 2, [0, 2600]), (128, 3, 1, [0, 3001]),
          (128, 5, 1, [0, 129, 3400]), (128, 4, 2, [0, 3500, 3503]), (64, 8, 1, [0, 3333])]


@pytest.mark.parametrize("d,hq,hkv,offsets", SHAPES)
def test_random_rows(d, hq, hkv, offsets):
    gen = torch.Generator(device="cuda").manual_seed(d + hq)
    n = offsets[-1]
    q, k, v = (torch.randn((n, h, d), generator=gen, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    out, lse, (want, wlse, spread, reach) = attend(q, k, v, offsets)
    bound = check_lse(lse, wlse, reach, d, offsets)
    # a key more or less moves ln sum by its probability, ~1 / n on average: the bound sees it
    rows = np.concatenate([np.arange(1, b - a + 1) for a, b in zip(offsets, offsets[1:])])
    assert (bound.max(1) < 1.0 / rows).all()
    check_out(out, want, spread, reach, d, offsets)
    # In the 2-norm: a rounding to BF16 of values m 2^e, m in [1, 2), is uniform within
    # 2^-8 2^e, so 2^-8 / sqrt(3) / rms(m) of them; rms(m) is 1.47 where their logarithms
    # are spread evenly and 1.53 where they are themselves; with 1.35 at least 0.00167.
    # The output takes one, and the probabilities' (independent, against V of random
    # signs) make another of the same size: 0.00236 together; FP32 sums stay below a
    # hundredth of that.  A key more or less in every row would be sqrt(1 / n), 0.014.
    assert np.linalg.norm(out - want) <= 0.0024 * np.linalg.norm(want)


@pytest.mark.parametrize("d,hq,hkv,offsets", SHAPES)
@pytest.mark.parametrize("at", ["own", "next", "any", "first"])
def test_one_key_that_outweighs_all(d, hq, hkv, offsets, at):
    """Keys 4 c_j, c_j of random signs; a query c_j has a score of 4 sqrt(d) there and
    4 N(0, 1) elsewhere.  The key is the row's own, the one behind it (which it does not
    see: the others stay as they are), any before it, or the sequence's first."""
    gen = torch.Generator(device="cuda").manual_seed(d + hq)
    rng = np.random.default_rng(d + hq)
    n = offsets[-1]
    signs = (torch.randint(0, 2, (n, hkv, d), generator=gen, device="cuda") * 2 - 1).to(torch.bfloat16)
    v = torch.randn((n, hkv, d), generator=gen, device="cuda").to(torch.bfloat16)
    row = np.arange(n)
    start = np.concatenate([np.full(b - a, a) for a, b in zip(offsets, offsets[1:])])
    key = {"own": row, "next": np.minimum(row + 1, n - 1), "first": start,
           "any": start + (rng.random(n) * (row - start + 1)).astype(np.int64)}[at]
    q = signs[torch.from_numpy(key).cuda()].repeat_interleave(hq // hkv, 1)
    out, lse, (want, wlse, spread, reach) = attend(q, signs * 4, v, offsets)
    check_lse(lse, wlse, reach, d, offsets)
    check_out(out, want, spread, reach, d, offsets)
