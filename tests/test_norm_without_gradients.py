"""clip_grad_norm of no gradients gives zero, a float32 where the parameters are; an optimizer's step gives none."""
import pytest
import torch

from rank_randomized_gradient_amd import AdamW, clip_grad_norm


@pytest.mark.parametrize("device", ["cpu", "meta", pytest.param("cuda", marks=pytest.mark.gpu)])
def test_zero_on_the_parameters_device(device):
    if device == "cuda" and not torch.cuda.is_available():
        pytest.skip("no GPU")
    p = torch.nn.Parameter(torch.zeros(5, dtype=torch.bfloat16, device=device))
    opt = AdamW([p])
    for norm in (clip_grad_norm([p], 1.0), clip_grad_norm(p, 1.0), clip_grad_norm(iter([p]), 1.0)):
        assert norm.shape == () and norm.dtype == torch.float32 and norm.device.type == device
        assert device == "meta" or float(norm) == 0
    assert opt.step(max_norm=1.0) is None and opt.step() is None and opt.steps == 2


def test_no_parameters():
    norm = clip_grad_norm([], 1.0)
    assert norm.shape == () and norm.dtype == torch.float32 and float(norm) == 0
