"""Lengths that do not fit the C ABI's 32 bits are refused by the binding: their
low bits alone are another call's (2^32 would be a bound of 0, which computes
nothing and says so to nobody)."""
import pytest
import torch

import quantized_paged_kv_write_gb300 as kvq

z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
FMT = kvq.CacheFormat("int8", "int8", "token_head", "token_head", 2, 64, 4)


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32, 2 ** 32 + 20, 2 ** 64 + 5, -2 ** 31 - 1, -2 ** 32 + 7])
def test_lengths_past_32_bits_are_refused(n):
    i = lambda *s: z(*s, t=torch.int32)  # noqa: E731
    q, k = z(5, 4, 64), z(5, 2, 64)
    calls = [lambda: kvq.kvq_prompt_attention(q, k, k, i(2), n, out=q, workspace=z(9, t=torch.uint8)),
             lambda: kvq.kvq_prompt_attention(q, k, k, i(2), n),
             lambda: kvq.kvq_prompt_attention_workspace_size(1, n, 4, 2),
             lambda: kvq.kvq_prompt_attention_workspace_size(n, 5, 4, 2),
             lambda: kvq.kvq_weigh_decode(z(2, 4, 64), FMT, {}, i(2, 4), i(2), n, z(2, 2, 64, t=torch.float32)),
             lambda: kvq.kvq_weigh_decode(z(2, 4, 64), FMT, {}, i(2, 4), i(2), n, z(2, 2, 64, t=torch.float32),
                                          out=z(2, 4, 64, t=torch.float32), workspace=z(9, t=torch.uint8)),
             lambda: kvq.kvq_weigh_decode_workspace_size(FMT, 2, 4, n),
             lambda: kvq.kvq_weigh_decode_workspace_size(FMT, n, 4, 60),
             lambda: kvq.kvq_evict_workspace_size(1, 2, n),
             lambda: kvq.kvq_evict_workspace_size(n, 2, 60)]
    for call in calls:
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_weights_of_rows_past_32_bits_are_refused():
    """(a row of 2^32 + 16 entries, without the memory for it)"""
    i = lambda *s: z(*s, t=torch.int32)  # noqa: E731
    wide = z(1, t=torch.float32).expand(1, 2, 2 ** 32 + 16)
    with pytest.raises(ValueError, match="32 bits"):
        kvq.kvq_evict_tokens(i(1), i(1), i(1, 4), FMT, {}, wide, i(1), kept_lens=i(1), workspace=z(9, t=torch.uint8))


def test_tables_of_rows_past_32_bits_are_refused():
    i = lambda *s: z(*s, t=torch.int32)  # noqa: E731
    wide, w = i(1).expand(1, 2 ** 32 + 4), z(1, 2, 64, t=torch.float32)
    with pytest.raises(ValueError, match="32 bits"):
        kvq.kvq_evict_tokens(i(1), i(1), wide, FMT, {}, w, i(1), kept_lens=i(1), workspace=z(9, t=torch.uint8))
    with pytest.raises(ValueError, match="32 bits"):
        kvq.kvq_weigh_decode(z(1, 4, 64), FMT, {}, wide, i(1), 60, w, out=z(1, 4, 64, t=torch.float32), workspace=z(9, t=torch.uint8))


def test_lengths_of_32_bits_reach_the_library():
    with pytest.raises(kvq.KvqError, match="unsupported"):
        kvq.kvq_prompt_attention_workspace_size(1, 2 ** 31 - 1, 4, 2)
    with pytest.raises(kvq.KvqError, match="invalid"):
        kvq.kvq_evict_workspace_size(1, 2, -2 ** 31)
