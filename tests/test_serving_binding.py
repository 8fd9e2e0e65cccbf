"""The answering path's binding: what it needs of PyTorch when it is imported.  CPU only."""

import importlib.util

import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab

NAMES = ("_cuda_getDevice", "_cuda_getCurrentRawStream", "_cuda_isCurrentStreamCapturing")


def test_import_needs_no_cuda_build(monkeypatch):
    """A PyTorch built without CUDA lacks these names."""
    for n in NAMES:
        monkeypatch.delattr(torch._C, n, raising=False)
    spec = importlib.util.spec_from_file_location(ab.__name__ + "_again", ab.__file__)
    mod = importlib.util.module_from_spec(spec)
    mod.__package__ = ab.__package__
    spec.loader.exec_module(mod)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mod.rope_fwd(torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16), None, None, None)
