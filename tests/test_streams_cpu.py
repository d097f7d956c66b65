"""Which stream a call's `stream` argument means, without a GPU."""

import torch

import bit_weight_gemm_amd as bw


def test_handles_become_the_streams_they_name(monkeypatch):
    """The handle 0 names the default stream; wrapped as any other it would become a new stream of torch's pool."""
    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

    default = Stream(0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: default)
    assert bw._on(None) is None
    own = Stream(4096)
    assert bw._on(own) is own
    assert bw._on(8192).cuda_stream == 8192
    assert bw._on(0) is default
