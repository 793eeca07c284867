"""What the Python binding of the operators around the linears refuses before it calls the library (no GPU needed)."""
from types import SimpleNamespace

import pytest
import torch

from epilogue_gemm_nvfp4_b200 import binding as B


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Its work would otherwise go to the current stream of the tensors' device."""
    monkeypatch.setattr(torch.cuda, "stream", lambda s: ("on", s))
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    t = SimpleNamespace(is_cuda=True, get_device=lambda: 0)
    same, other = (SimpleNamespace(device=torch.device("cuda", i)) for i in (0, 1))
    assert B._here(same, t) == ("on", same)
    assert B._here(None, t) is None
    with pytest.raises(ValueError):
        B._here(other, t)
