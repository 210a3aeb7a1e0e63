"""CPU checks of how the calls on adapters and gradients reach the library."""
import pytest
import torch

import orthogonal_fine_tuning_amd as oft


class _Stream:
    cuda_stream = 0x5000


@pytest.mark.parametrize("private", [True, False])
def test_stream_and_device_without_torchs_private_calls(monkeypatch, private):
    """The current stream and device are asked for below torch.cuda's objects
    where torch offers that, and through them where it does not."""
    asked = []
    names = ("_cuda_getCurrentRawStream", "_cuda_getDevice")
    if private:
        monkeypatch.setattr(torch._C, names[0], lambda dev: asked.append(("raw", dev)) or 0x6000, raising=False)
        monkeypatch.setattr(torch._C, names[1], lambda: 0, raising=False)
    else:
        for name in names:
            monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: asked.append(("public", dev)) or _Stream())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(oft, "_ASK", [])
    with pytest.raises(oft.OftError):  # (a negative count: refused before the stream is looked at)
        oft._launch("oft_grad_sumsq", 0, None, -1, None, None, oft.OFT_DT_F32, None, None, 0)
    assert asked == [("raw" if private else "public", 0)]
