"""What kvq_prompt_attention reports of bad offsets: their order and range alone
(KVQ_DEVERR_GROUP_RANGE), whatever lengths they would make."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offsets,bound", [([0, 100, 301], 300), ([0, 301], 400), ([0, 2 ** 31 - 1, 100], 300), ([0, 250, 100], 200),
                                           ([-(2 ** 31), 2 ** 31 - 1], 300), ([-5, 300], 400), ([0, 10, 200, 150, 300], 100)])
def test_bad_offsets_say_nothing_of_lengths(offsets, bound):
    from quantized_paged_kv_write_gb300 import build
    build.build()
    import quantized_paged_kv_write_gb300 as kvq
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn((300, h, 64), generator=gen, device="cuda").to(torch.bfloat16) for h in (2, 1, 1))
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    kvq.kvq_prompt_attention(q, k, v, torch.tensor(offsets, dtype=torch.int32, device="cuda"), bound, out=out, lse=lse)
    assert kvq.kvq_device_errors() == kvq.DEVERR_GROUP_RANGE
    assert bool((out == 7).all()) and bool((lse == 7).all())
