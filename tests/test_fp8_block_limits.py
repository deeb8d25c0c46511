"""Limits of the FP8 block-scale calls on the host: head counts past 32-bit offsets are refused, and the
binding finds its way without torch's private shortcuts."""
import types

import torch

P = 1 << 20  # an aligned address that no refused call dereferences


def test_prefill_refuses_heads_past_its_offsets(libpa):
    args = lambda hq, hkv, n: (P, P, P, P, P, P, 4, P, P, n, 20, 9, hq, hkv, 128, 16, 8, 0.1, P, 1, None)  # noqa: E731
    run = libpa.lib().pa_prefill_fp8_block
    assert run(*args(1 << 17, 1 << 17, 3)) == libpa.PA_ERR_ARG
    assert run(*args(1 << 17, 1 << 17, 0)) == libpa.PA_ERR_ARG
    assert run(*args(65536, 65536, 0)) == libpa.PA_OK  # (no sequences)


def test_the_binding_without_torchs_shortcuts(libpa, monkeypatch):
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    t = libpa._Torch()
    assert t.current_device is torch.cuda.current_device
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: types.SimpleNamespace(cuda_stream=77 + dev))
    assert t.raw_stream(2) == 79
