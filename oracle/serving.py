"""Oracle: causal attention over packed prompts, the attention weights of cached
tokens, and eviction by them (test infrastructure; see the package docstring).

Attention is softmax(q·kᵀ / sqrt(d)) · V with GQA groups ("PidokuInfra 12 KV
Cache Quantization", §5; "KV Cache Quantization" glossary), everything in
float64.  The pages have no eviction: which tokens stay and where they go is the
library's stated contract, restated here one token at a time.
"""
from __future__ import annotations

import functools
import math

import numpy as np

from .attention import _sequence_rows
from .quantize import OracleCache, bf16_bits_to_f32, dequantize_cache_rows

BLOCK = 16


def prompt_attention_fp64(q, k, v, offsets):
    """q float64 [N, Hq, d], k, v [N, H, d], offsets [S + 1].  Returns (out, lse,
    spread, reach): [N, Hq, d], [N, Hq], sum p |v| [N, Hq, d] and the largest sum
    |q_i k_i| / sqrt(d) of the row's scores [N, Hq] (what rounding errors scale
    with); NaN outside every sequence."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    out, spread = np.full((n, hq, d), np.nan), np.full((n, hq, d), np.nan)
    lse, reach = np.full((n, hq), np.nan), np.full((n, hq), np.nan)
    for a, b in zip(offsets, offsets[1:]):
        for h in range(hq):
            kk, vv = k[a:b, h // g], v[a:b, h // g]
            z = q[a:b, h] @ kk.T / math.sqrt(d)
            z = np.where(np.tri(b - a, dtype=bool), z, -np.inf)
            m = z.max(1, keepdims=True) if b > a else np.zeros((0, 1))
            p = np.exp(z - m)
            s = p.sum(1, keepdims=True)
            p /= s
            out[a:b, h], spread[a:b, h] = p @ vv, p @ np.abs(vv)
            lse[a:b, h] = (m + np.log(s))[:, 0]
            big = np.abs(q[a:b, h]) @ np.abs(kk).T / math.sqrt(d)
            reach[a:b, h] = np.where(np.tri(b - a, dtype=bool), big, 0).max(1) if b > a else 0
    return out, lse, spread, reach


def attention_weights_fp64(cache: OracleCache, q_bits, tables, context_lens, length):
    """Per (sequence, kv head, position): the sum over the kv head's query heads
    of the softmax, and the largest sum |q_i k_i| / sqrt(d) of any of the
    sequence's scores.  [B, H, length], [B]."""
    bsz, hq, d = q_bits.shape
    h, g = cache.num_kv_heads, hq // cache.num_kv_heads
    got, reach = np.zeros((bsz, h, length)), np.zeros(bsz)
    for b in range(bsz):
        n = int(context_lens[b])
        if n == 0:
            continue
        blocks, offs = _sequence_rows(cache, tables[b], n)
        k = dequantize_cache_rows(cache, "k", blocks, offs)
        q = bf16_bits_to_f32(q_bits[b]).astype(np.float64)
        if cache.rotation is not None:
            from .rotation import rotate_query_fp64
            q = rotate_query_fp64(q, cache.rotation)
        for x in range(hq):
            z = k[:, x // g] @ q[x] / math.sqrt(d)
            p = np.exp(z - z.max())
            got[b, x // g, :n] += p / p.sum()
            reach[b] = max(reach[b], float((np.abs(k[:, x // g]) @ np.abs(q[x])).max()) / math.sqrt(d))
    return got, reach


def _heavier(x, y):
    """Whether weight x goes before y (NaN counts as the heaviest)."""
    return (not math.isnan(y)) if math.isnan(x) else (not math.isnan(y) and x > y)


def evict_tokens(keep, recent, pinned, context_lens, tables, arrays, weights, refs=None):
    """arrays: cache arrays [num_blocks, 16, H, ...]; arrays and weights [R, H,
    positions] are updated in place.  Returns kept_lens."""
    num_blocks = arrays[0].shape[0]
    rows, heads, length = weights.shape
    kept = [int(n) for n in context_lens]
    for r in range(rows):
        n, k = int(context_lens[r]), int(keep[r])
        if n < 0 or n > min(length, tables.shape[1] * BLOCK) or min(k, int(recent[r]), int(pinned[r])) < 0 or n <= k:
            continue
        w = min(int(recent[r]), k)
        p = min(int(pinned[r]), k - w)
        ids = [int(x) for x in tables[r, :-(-n // BLOCK)]]
        if any(x not in range(num_blocks) for x in ids):
            continue
        if refs is not None and p < k and any(refs[x] != 1 for x in ids[p // BLOCK:-(-k // BLOCK)]):
            continue
        kept[r] = k
        for h in range(heads):
            x = weights[r, h]
            order = list(range(p, n - w))
            order.sort(key=functools.cmp_to_key(
                lambda i, j: -1 if _heavier(x[i], x[j]) else 1 if _heavier(x[j], x[i]) else i - j))
            stay = set(order[:k - w - p])
            places = [i for i in range(p, k - w) if i not in stay]
            tokens = sorted(i for i in stay if i >= k - w)
            assert len(places) == len(tokens)
            places += range(k - w, k)
            tokens += range(n - w, n)
            at = lambda i: (ids[i // BLOCK], i % BLOCK, h)  # noqa: E731
            for y in arrays:
                old = [y[at(i)].copy() for i in tokens]
                for i, v in zip(places, old):
                    y[at(i)] = v
            old = [x[i] for i in tokens]
            for i, v in zip(places, old):
                x[i] = v
            x[k:n] = 0
    return np.array(kept, np.int32)
