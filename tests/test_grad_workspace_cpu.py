"""alloc_grad_workspace takes what moe_grad_norm and moe_clip_grads take: any iterable of tensors."""
import pytest
import torch

from sparse_mixture_experts_17_b200 import moe as M


@pytest.mark.parametrize("of", [list, tuple, iter, lambda ts: (t for t in ts), lambda ts: dict(enumerate(ts)).values()])
@pytest.mark.parametrize("n", [0, 1, 3])
def test_any_iterable(of, n):
    ws = M.alloc_grad_workspace(of([torch.zeros(4) for _ in range(n)]), device="cpu")
    assert ws.numel() == M.MOE_GRAD_WS_BYTES and ws.device.type == "cpu"
