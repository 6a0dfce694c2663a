"""kvq_prefix_decode at the ends of what its arguments allow."""
import pytest
import torch

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
