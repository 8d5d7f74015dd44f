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


@pytest.mark.parametrize("row,head", [(512, 64), (64, 640), (0, 0)])
def test_an_empty_batch_of_a_strided_view_is_an_empty_call(lib, row, head):
    """torch gives every empty tensor the address 0, so x and a fresh y look like one tensor with different strides: no
    rotation in place, and nothing to refuse."""
    args = (0, 2, 64, 32, 2, 8)
    assert lib.flashnorm_rope(NULL, P, NULL, NULL, *args, row, head, 128, 64, 0, 0, 0, NULL) == fn.FN_OK
    assert lib.flashnorm_rope(P, P, P, P, *args, row, head, 128, 64, 0, 0, 0, NULL) == fn.FN_OK
    # with rows it still is one
    assert lib.flashnorm_rope(P, P, P, P, 4, *args[1:], row, head, 128, 64, 0, 0, 0, NULL) == fn.FN_ERR_INVALID_ARG


@pytest.mark.gpu
def test_empty_batch_of_a_strided_view_on_the_gpu():
    qkv = torch.randn(5, 6, 32, device="cuda")[:, 1:4]
    cs = fn.flashnorm_rope_table_scaled(8, 32)
    pos = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert fn.flashnorm_rope(qkv[:0], cs, pos[:0]).shape == (0, 3, 32)
    fn.flashnorm_check_device_error()
