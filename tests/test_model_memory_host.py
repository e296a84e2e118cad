"""Outputs of the norm in front of a block that are given in the memory of its inputs: the
same view where the call may run in place, else refused before anything is launched."""
import pytest
import torch

import mamba_ssd_forward_gb300 as ssd
from test_model_host import OnDevice, abi, far  # noqa: F401

B16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def wide(*shape, dtype=torch.float32):
    """The left half of rows twice as wide, and a dense tensor at the same address."""
    base = far(shape[0], 2 * shape[1], dtype=dtype)
    return base[:, :shape[1]], base.reshape(-1)[:shape[0] * shape[1]].reshape(shape)


def refusals():
    x, r, w = far(4, 64, dtype=B16), far(4, 64), far(64)
    xw, xd = wide(4, 64, dtype=B16)
    rw, rd = wide(4, 64)
    total = far(4, 64)
    f, q = ssd.add_norm_forward, ssd.add_norm_quantized

    def bytes_of(t):
        return t.reshape(-1).view(E4M3)[:4 * 64].reshape(4, 64)

    return {
        "y over x": (lambda: f(xw, r, w, y=xd), "y must be x itself"),
        "total over residual": (lambda: f(x, rw, w, total=rd), "total must be residual itself"),
        "quantised total over residual": (lambda: q(x, rw, w, total=rd), "total must be residual"),
        "q over x": (lambda: q(x, r, w, q=bytes_of(x)), "q must not be the memory of x"),
        "q over residual": (lambda: q(x, r, w, q=bytes_of(r)), "q must not .* of residual"),
        "q over total": (lambda: q(x, r, w, q=bytes_of(total), total=total), "q must not .* of total"),
        "scales over residual": (lambda: q(x, r, w, block=0, scales=r.reshape(-1)[:4].reshape(4, 1)),
                                 "scales must not .* of residual"),
        "scales over total": (lambda: q(x, r, w, block=0, total=total,
                                        scales=total.reshape(-1)[:4].reshape(4, 1)),
                              "scales must not .* of total"),
    }


@pytest.fixture
def on_device(abi, monkeypatch):  # noqa: F811
    """Outputs on the tensors' device, which is not the current one."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    real = torch.empty

    def empty(*a, **k):
        k.pop("device", None)
        return real(*a, **k).as_subclass(OnDevice)

    monkeypatch.setattr(torch, "empty", empty)


@pytest.mark.parametrize("name", list(refusals()))
def test_overlaps_are_refused(on_device, name):
    call, words = refusals()[name]
    with pytest.raises(ValueError, match=words):
        call()


def test_the_same_view_is_not(on_device):
    """These pass the checks and fail at the next one, the device's."""
    xw, xd = wide(4, 64, dtype=B16)
    rw, rd = wide(4, 64)
    one, w = wide(1, 64, dtype=B16), far(64)
    for call in (lambda: ssd.add_norm_forward(xw, rw, w, y=xw, total=rw),
                 lambda: ssd.add_norm_forward(xd, rd, w, y=xd, total=rd),
                 lambda: ssd.add_norm_forward(one[0], far(1, 64), w, y=one[1]),  # one row: the same
                 lambda: ssd.add_norm_quantized(xw, rw, w, total=rw)):
        with pytest.raises(ValueError, match="current device"):
            call()
