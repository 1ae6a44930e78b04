"""What the attention-side calls take for a stream, without a GPU."""
import pytest
import torch

import fp4_activation_sparse_b200 as S


class Wrapper:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle
        if device is not None:
            self.device = device


DEVICE = torch.device("cuda", 0)


@pytest.mark.parametrize("stream,handle", [(0, 0), (0x5550, 0x5550), (Wrapper(0x40), 0x40), (Wrapper(0x40, "cuda:0"), 0x40),
                                           (Wrapper(0, DEVICE), 0), (Wrapper(0x40, "cuda"), 0x40), (Wrapper(0x40, 0), 0x40)])
def test_handles(stream, handle):
    assert S._stream_handle(stream, DEVICE) == handle


@pytest.mark.parametrize("stream", [Wrapper(0x40, "cuda:1"), Wrapper(0x40, torch.device("cuda", 3)), Wrapper(None), "main", object(),
                                    Wrapper(0x40, "somewhere"), Wrapper(0x40, "cpu"), Wrapper(0x40, 1)])
def test_refused(stream):
    """A stream of another device would be dropped in silence; something else is no stream."""
    for call in (S._stream_handle, S._on_stream):
        with pytest.raises(S.SharqError) as e:
            call(stream, DEVICE)
        assert e.value.status == S.SHARQ_ERR_INVALID_ARG


def test_host_tensors_are_refused_with_a_stream_too():
    y = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(S.SharqError):
        S.sharq_norm_residual(y, y, stream=0)
