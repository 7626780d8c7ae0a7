"""A caller's workspace on another device than the tensors (CPU only)."""
import pytest
import torch

from rank_randomized_gradient_amd import rgc


def test_a_workspace_of_another_device_is_refused():
    """Its address would go to the kernels as it is."""
    ws = rgc.Workspace(torch.device("cpu"))
    with pytest.raises(rgc.RgcError):
        rgc._scratch(ws, 1 << 12, torch.device("cuda", 0))
    assert ws.buf.numel() == 0
