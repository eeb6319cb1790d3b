"""The linear products' activations far from zero (the derivative of gelu's tanh form where z^2
leaves fp32, the lower tail of gelu), and the bias gradients of long groups."""
import math

import pytest
import torch

from sparse_mixture_experts_17_b200 import moe as M
from test_gpu_linear import ACTS, BF16, F32, U, assert_within, sizes_to_offsets, slope64

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


def test_tail_of_gelu_past_six():
    """gelu(z) and its derivative for z from -12.9 to -6 keep their relative accuracy: Phi to 2^-10 (its
    logarithm is a cubic there, 6.5e-4 off at most), and one rounding to bf16. Below, where Phi is
    under fp32's smallest normal number, it counts as 0."""
    z = torch.linspace(-12.9, -6, 1024, device="cuda").to(BF16)
    n = z.numel()
    W = torch.zeros(n, 8, dtype=BF16, device="cuda")
    W[:, 0] = z
    x = torch.zeros(3, 8, dtype=BF16, device="cuda")
    x[:, 0] = 1.0
    y = torch.empty(3, n, dtype=BF16, device="cuda")
    M.moe_linear_forward(M.make_linear(3, 8, n, act=M.MOE_ACT_GELU), x, None, W, None, None, y)
    z64 = z.double()
    Phi = 0.5 * torch.special.erfc(-z64 * math.sqrt(0.5))      # torch's ndtr is (1 + erf) / 2: 1e-16 off here
    ref = (z64 * Phi).expand(3, -1)
    assert_within(y, ref, (U + 2.0 ** -10) * ref.abs(), "gelu")
    db, _ = slopes(z, "gelu")
    ref = Phi + z64 * torch.exp(-0.5 * z64 * z64) / math.sqrt(2 * math.pi)
    assert_within(db, ref, 2.0 ** -10 * ref.abs(), "derivative of gelu")
    far = torch.tensor([-13.5, -14.0, -20.0, -100.0, -1e19, -1e30, -3e38, -3.38e38], device="cuda").to(BF16)
    W = torch.zeros(8, 8, dtype=BF16, device="cuda")
    W[:, 0] = far
    y = torch.empty(3, 8, dtype=BF16, device="cuda")
    M.moe_linear_forward(M.make_linear(3, 8, 8, act=M.MOE_ACT_GELU), x, None, W, None, None, y)
    assert bool((y.abs().double() <= 2.0 ** -122).all())


@pytest.mark.parametrize("sizes", [[1 << 20], [1 << 19, 0, 33, 1 << 20]])
def test_bias_gradients_of_long_groups(sizes):
    """The bias gradient of a group of a million rows, with terms of one sign and one value (what the mean of
    a loss gives), keeps fp32's bits: at most 12 fp32 additions in a row, and fp64 from there. dz carries
    the derivative's 7e-7 (1 + |z|) = 1.4e-6 of dy, the product's rounding and the sums' 13."""
    off = sizes_to_offsets(sizes)
    rows, E = off[-1], len(sizes)
    z = torch.ones(rows, 8, dtype=BF16, device="cuda")
    dy = torch.full((rows, 8), 0.1, dtype=BF16, device="cuda")
    db = torch.empty(E, 8, dtype=F32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = M.make_linear(rows, 8, 8, E=E, act=M.MOE_ACT_SILU)
    M.moe_linear_backward(s, None, torch.tensor(off, dtype=torch.int32, device="cuda"), None, z, dy, None, None, db,
                          status, M.alloc_linear_workspace(s))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    slope = float(slope64(torch.ones(1, dtype=torch.float64), "silu"))
    ref = torch.tensor(sizes, dtype=torch.float64, device="cuda")[:, None] * float(dy[0, 0]) * slope
    assert_within(db, ref.expand(E, 8), (1.4e-6 / slope + 14 * 2.0 ** -24) * ref, "db")
