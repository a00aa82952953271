"""GPU tests of ``stream_workspace``: one for each device and stream, however the
device is named."""
import pytest
import torch

from weight_only_int4_unpack_amd import w4a16 as W

pytestmark = pytest.mark.gpu


def test_a_device_without_an_index_is_the_current_one():
    here = torch.device("cuda", torch.cuda.current_device())
    a = W.stream_workspace(torch.device("cuda"), 100000)
    assert a.numel() >= 100000 and a.device == here and a.data_ptr() == W.stream_workspace(here, 100000).data_ptr()
    assert not a[:W.WORKSPACE_COUNTER_BYTES].any()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = W.stream_workspace(torch.device("cuda"), 100000)
        assert b.data_ptr() != a.data_ptr() and b.data_ptr() == W.stream_workspace(here, 100000).data_ptr()
    assert W.stream_workspace(torch.device("cuda"), 0) is None
