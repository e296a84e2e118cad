"""Host side of the calls around the scan (no GPU needed): what they refuse by
name before anything is launched, and what they ask of the library."""
import pytest
import torch

import mamba_ssd_forward_gb300 as ssd


class OnDevice1(torch.Tensor):
    """A host tensor that says it is on cuda:1; never dereferenced."""

    is_cuda = True
    device = torch.device("cuda", 1)

    def get_device(self):
        return 1


def far(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice1)


def _calls():
    x, w, tok = far(2, 5, 8), far(8, 4), far(2, 8)
    A, B = far(8, 4), far(2, 5, 1, 4)
    big = far(1 << 20, dtype=torch.uint8)
    x4, dt, B4, D1 = far(1, 64, 2, 64), far(1, 64, 2), far(1, 64, 1, 64), far(2)
    return {
        "conv": lambda: ssd.causal_conv_forward(x, w, y=far(2, 5, 8), return_final_state=False),
        "conv_step": lambda: ssd.causal_conv_step(tok, w, None, far(2, 3, 8), y=far(2, 8)),
        "scan": lambda: ssd.selective_scan_forward(x, x, A, B, B, y=far(2, 5, 8), workspace=big,
                                                   return_final_state=False),
        "scan_step": lambda: ssd.selective_scan_step(tok, tok, A, B[:, 0], B[:, 0], None, None,
                                                     None, far(2, 8, 4), y=far(2, 8)),
        "norm": lambda: ssd.gated_norm_forward(x, far(8), gate="none", y=far(2, 5, 8)),
        "forward": lambda: ssd.forward(x4, dt, D1, B4, B4, chunk=64, y=far(1, 64, 2, 64),
                                       workspace=big, return_final_state=False),
        "decode_step": lambda: ssd.decode_step(x4[:, 0], dt[:, 0], D1, B4[:, 0], B4[:, 0], None,
                                               far(1, 2, 64, 64), y=far(1, 2, 64)),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    """The library launches on the current device, cuda:0 here."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="cuda:1.*current.*cuda:0"):
        _calls()[name]()
