"""The linear products' activations far from zero: the derivative of gelu's tanh form where
z^2 leaves fp32."""
import pytest
import torch

from sparse_mixture_experts_17_b200 import moe as M
from test_gpu_linear import ACTS, BF16, F32, U, assert_within, slope64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_17_b200 import build
    build.build()


def slopes(z, act):
    """act'(z) for a row of z, as the two fp32 sums of a backward call give it (dy = 1), and its dz in
    bf16, read off dx with W the identity."""
    n = z.numel()
    zz = z[None].expand(2, n).contiguous()
    dy = torch.ones(2, n, dtype=BF16, device="cuda")
    W = torch.eye(n, dtype=BF16, device="cuda")
    dx, db = torch.empty(2, n, dtype=BF16, device="cuda"), torch.empty(n, dtype=F32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = M.make_linear(2, n, n, act=ACTS[act])
    M.moe_linear_backward(s, None, None, W, zz, dy, dx, None, db, status, M.alloc_linear_workspace(s))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return db / 2, dx


@pytest.mark.parametrize("act", [a for a in ACTS if a != "none"])
def test_derivatives_of_huge_values(act):
    """bf16 reaches 3.4e38: z^2 and z^3 leave fp32, the derivative is 0 or 1 all the same. From 16 on it is
    within 2^-19 of its limit for every activation (silu: 16 e^-16 = 2^-19.1), and the formulas are
    good to 2^-18 there."""
    big = torch.tensor([16.0, 100.0, 1e4, 1e12, 1.8e19, 1.9e19, 1e20, 1e25, 1e30, 1e38, 2e38, 3.3e38], device="cuda")
    z = torch.cat([big, -big]).to(BF16)
    db, dx = slopes(z, act)
    ref = slope64(z.double(), act)
    assert bool(torch.isfinite(ref).all())
    assert_within(db, ref, torch.full_like(ref, 2.0 ** -18), "derivative")
    assert_within(dx[0], ref, U * ref.abs() + 2.0 ** -17, "dz")
