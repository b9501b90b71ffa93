"""The stream that the binding hands to the library, with stand-ins for torch's: the
default stream of a device that is not the current one is refused (its handle is
0, the current device's), any other stream knows its device."""
import types

import pytest
import torch

import bit_block_quantized_nibble_amd as qbn


@pytest.mark.parametrize("current,device,handle,ok", [(0, 0, 0, True), (1, 1, 0, True), (0, 1, 0x1234, True), (0, 1, 0, False),
                                                      (1, 0, 0, False)])
def test_default_stream_of_another_device_is_refused(monkeypatch, current, device, handle, ok):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=handle))
    prepared = qbn.Prepared(lambda stream: 0, (), "nothing", torch.device("cuda", device), None)
    if ok:
        assert (qbn._stream(torch.device("cuda", device)).value or 0) == handle
        prepared()
    else:
        with pytest.raises(ValueError, match="not the current device"):
            qbn._stream(torch.device("cuda", device))
        with pytest.raises(ValueError, match="not the current device"):
            prepared()
