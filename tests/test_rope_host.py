"""Host side of the rotary calls that needs no GPU: what is refused, and what is not, before anything is launched."""

import ctypes

import pytest
import torch

import rmsnorm_linear_projection_fold_b200 as fn

NULL = ctypes.c_void_p(None)
P = ctypes.c_void_p(1 << 20)


@pytest.fixture(scope="module")
def lib():
    from rmsnorm_linear_projection_fold_b200 import build

    build.build()
    return fn.load_library()


@pytest.mark.parametrize("device", ["cpu", torch.device("cpu"), "meta"])
def test_table_is_made_on_a_cuda_device_only(monkeypatch, device):
    """A table in host memory would be an address that the kernel must not write to: refused before the library is called."""
    calls = []
    monkeypatch.setattr(fn, "_invoke_on", lambda *a, **k: calls.append(a))
    monkeypatch.setattr(fn, "_stream_ptr", lambda t: 0)
    with pytest.raises(ValueError, match="CUDA"):
        fn.flashnorm_rope_table_scaled(8, 4, device=device)
    assert not calls
