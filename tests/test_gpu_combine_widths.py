"""moe_combine_rows and its gradient on rows of every width that a linear product can write (multiples of 8
from 8 on), with the shape's unused fields left at 0. Bounds as in test_gpu_combine_rows.py."""
import pytest
import torch

from sparse_mixture_experts_17_b200 import moe as M
from test_gpu_combine_rows import BF16, F32, I32, U, make, ref_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_17_b200 import build
    build.build()


@pytest.mark.parametrize("T,d,k,E", [(1, 8, 1, 1), (5, 8, 16, 16), (3, 24, 2, 8), (64, 72, 3, 5), (1000, 200, 2, 8),
                                     (17, 1000, 8, 128), (300, 1288, 4, 4), (9, 16392, 2, 2), (2, 65536, 5, 7)])
def test_widths(T, d, k, E):
    s = M.make_shape(T, d, 0, E, k)
    slot, y, w, R, used = make(T, d, k, 0.3, seed=T + d)
    status = torch.zeros(1, dtype=I32, device="cuda")
    for ww in (w, None):
        for res in (R, None):
            out = torch.full((T, d), 9.0, dtype=BF16, device="cuda")
            M.moe_combine_rows(s, y, slot, ww, res, out, status)
            ref, mag = ref_out(slot, y, ww, res)
            assert bool(((out.double() - ref).abs() <= U * ref.abs() + (k + 1) * 2.0 ** -24 * (1 + U) * mag).all())
    dout = torch.randn(T, d, device="cuda").to(BF16)
    dy = torch.full((T * k, d), 5.0, dtype=BF16, device="cuda")
    dw = torch.full((T, k), 5.0, dtype=F32, device="cuda")
    M.moe_combine_rows_backward(s, dout, y, slot, w, dy, dw, status)
    keep = slot >= 0
    rows = torch.where(keep.unsqueeze(-1), y[slot.clamp(min=0).long()].double(), 0.0)
    prod = dout.double().unsqueeze(1) * rows
    assert bool(((dw.double() - prod.sum(-1)).abs() <= (d + 8) * 2.0 ** -24 * prod.abs().sum(-1)).all())
    ref = (w.double().unsqueeze(-1) * dout.double().unsqueeze(1))[keep]
    assert bool(((dy[slot[keep].long()].double() - ref).abs() <= (U + 2.0 ** -22) * ref.abs()).all())
    assert bool((dy[~used] == 5.0).all()) and int(status.item()) == 0


def test_rows_of_a_linear_product():
    """Rows of 200 values, as moe_linear_forward writes them, combined."""
    T, k, E, di, do = 60, 2, 4, 64, 200
    g = torch.Generator("cuda").manual_seed(2)
    rnd = lambda *n: torch.randn(n, generator=g, device="cuda").to(BF16)
    off = torch.tensor([0, 50, 50, 90, T * k], dtype=I32, device="cuda")
    y, status = torch.empty(T * k, do, dtype=BF16, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    M.moe_linear_forward(M.make_linear(T * k, di, do, E=E), rnd(T * k, di), off, rnd(E, do, di), None, None, y, None, status)
    slot = torch.randperm(T * k, generator=g, device="cuda").reshape(T, k).to(I32)
    w = torch.rand(T, k, generator=g, device="cuda")
    out = torch.empty(T, do, dtype=BF16, device="cuda")
    M.moe_combine_rows(M.make_shape(T, do, 0, E, k), y, slot, w, None, out, status)
    ref, mag = ref_out(slot, y, w, None)
    assert bool(((out.double() - ref).abs() <= U * ref.abs() + (k + 1) * 2.0 ** -24 * (1 + U) * mag).all())
    assert int(status.item()) == 0
