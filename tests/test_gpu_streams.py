"""The attention-side calls on streams given in each of their forms."""
import pytest
import torch

from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu


class Wrapper:
    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.mark.parametrize("form", ["object", "handle", "wrapper", "default", "default handle", "legacy handle"])
def test_a_call_waits_for_the_work_of_its_stream(form):
    """The input is written late on the stream named, and by another stream's call nobody would wait for it."""
    S = require_gpu()
    side = torch.cuda.default_stream() if "default" in form or "legacy" in form else torch.cuda.Stream()
    given = {"object": side, "handle": side.cuda_stream, "wrapper": Wrapper(side), "default": side, "default handle": 0, "legacy handle": 1}[form]
    y = torch.randn(64, 1024, device="cuda").bfloat16()
    zero, late = torch.zeros_like(y), torch.zeros_like(y)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about ten milliseconds
        late.copy_(y)
    r, _ = S.sharq_norm_residual(late, zero, stream=given)
    torch.cuda.synchronize()
    assert torch.equal(r, y)
