"""A call's stream has to be of its tensors' device (stand-ins: no GPU is needed)."""

from types import SimpleNamespace

import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N


def test_a_stream_of_another_device_is_refused():
    stream = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=64)
    with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cuda:0"):
        N._stream(torch.device("cuda", 0), stream)
    assert N._stream(torch.device("cuda", 1), stream) == 64
