"""The stream that calls without one go to: torch's current stream, by its raw
handle where torch offers that and through its Stream object where not."""
import pytest
import torch

import q8_block_quantized_matvec_gb300 as q8d


@pytest.mark.parametrize("missing", [None, "_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_current_stream(monkeypatch, missing):
    current = {"device": 0, "handles": {0: 0x10, 1: 0x20}}

    class Stream:
        cuda_stream = property(lambda self: current["handles"][current["device"]])

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: current["handles"][d], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current["device"], raising=False)
    if missing:
        monkeypatch.delattr(torch._C, missing)
    monkeypatch.setattr(q8d, "_raw_stream", None)
    monkeypatch.setattr(q8d, "_device", None)
    assert q8d._stream(None) == 0x10
    current["handles"][0] = 0x30          # another stream made current
    assert q8d._stream(None) == 0x30
    current["device"] = 1                 # another device
    assert q8d._stream(None) == 0x20
    assert q8d._stream(Stream()) == 0x20 and q8d._stream(0x99) == 0x99
