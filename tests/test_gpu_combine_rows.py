"""moe_combine_rows and its gradient against fp64; dropped assignments, all
dropped, one slot to sixteen, odd widths, rows behind the kept ones.

Bounds: out is a sum of k + 1 fp32 terms rounded once to bf16 (2^-8 of the
value, and (k + 1) 2^-24 of the terms' magnitudes); dy one product and one
rounding; dw a sum of d exact products of bf16 values, (d + 8) 2^-24 of their
magnitudes."""
import pytest
import torch

from sparse_mixture_experts_17_b200 import moe as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_17_b200 import build
    build.build()


def make(T, d, k, drop, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    n = T * k
    perm = torch.randperm(n, generator=g, device="cuda").to(I32).reshape(T, k)
    dropped = torch.rand(T, k, generator=g, device="cuda") < drop
    slot = torch.where(dropped, torch.full_like(perm, -1), perm)
    y = torch.randn(n, d, generator=g, device="cuda").to(BF16)
    used = torch.zeros(n, dtype=torch.bool, device="cuda")
    used[perm[~dropped].long()] = True
    y[~used] = float("nan")               # rows that no slot names
    w = torch.rand(T, k, generator=g, device="cuda")
    R = torch.randn(T, d, generator=g, device="cuda").to(BF16)
    return slot, y, w, R, used


def ref_out(slot, y, w, R):
    keep = slot >= 0
    rows = torch.where(keep.unsqueeze(-1), y[slot.clamp(min=0).long()].double(), 0.0)
    ww = torch.ones_like(slot, dtype=torch.float64) if w is None else w.double()
    terms = ww.unsqueeze(-1) * rows
    out, mag = terms.sum(1), terms.abs().sum(1)
    return (out, mag) if R is None else (out + R.double(), mag + R.double().abs())


@pytest.mark.parametrize("T,d,k,E", [(1, 128, 1, 8), (1, 4096, 2, 8), (2, 7168, 8, 256), (3, 128, 16, 16),
                                     (17, 384, 3, 5), (33, 256, 5, 9), (100, 2048, 8, 128),
                                     (257, 640, 7, 7), (1000, 1152, 2, 8), (4099, 128, 4, 4)])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_forward_and_backward(T, d, k, E, drop):
    s = M.make_shape(T, d, 128, E, k)
    slot, y, w, R, used = make(T, d, k, drop, seed=T + k)
    status = torch.zeros(1, dtype=I32, device="cuda")
    for ww in (w, None):
        for res in (R, None):
            out = torch.full((T, d), 9.0, dtype=BF16, device="cuda")
            M.moe_combine_rows(s, y, slot, ww, res, out, status)
            ref, mag = ref_out(slot, y, ww, res)
            err = (out.double() - ref).abs()
            assert bool((err <= U * ref.abs() + (k + 1) * 2.0 ** -24 * (1 + U) * mag).all())
    alias = R.clone()
    M.moe_combine_rows(s, y, slot, w, alias, alias, status)
    out = torch.empty_like(R)
    M.moe_combine_rows(s, y, slot, w, R, out, status)
    assert torch.equal(alias, out)
    dout = torch.randn(T, d, device="cuda").to(BF16)
    dy = torch.full((T * k, d), 5.0, dtype=BF16, device="cuda")
    dw = torch.full((T, k), 5.0, dtype=F32, device="cuda")
    M.moe_combine_rows_backward(s, dout, y, slot, w, dy, dw, status)
    keep = slot >= 0
    rows = torch.where(keep.unsqueeze(-1), y[slot.clamp(min=0).long()].double(), 0.0)
    prod = dout.double().unsqueeze(1) * rows
    assert bool(((dw.double() - prod.sum(-1)).abs() <= (d + 8) * 2.0 ** -24 * prod.abs().sum(-1)).all())
    ref = (w.double().unsqueeze(-1) * dout.double().unsqueeze(1))[keep]
    got = dy[slot[keep].long()].double()
    assert bool(((got - ref).abs() <= (U + 2.0 ** -22) * ref.abs()).all())
    assert bool((dy[~used] == 5.0).all())
    # either output alone, and weights of one
    dy1, dw1 = torch.full_like(dy, 5.0), torch.full_like(dw, 5.0)
    M.moe_combine_rows_backward(s, dout, None, slot, w, dy1, None, status)
    M.moe_combine_rows_backward(s, dout, y, slot, None, None, dw1, status)
    assert torch.equal(dy1, dy) and torch.equal(dw1, dw)
    M.moe_combine_rows_backward(s, dout, None, slot, None, dy1, None, status)
    assert torch.equal(dy1[slot[keep].long()], dout.unsqueeze(1).expand(T, k, d)[keep])
    assert int(status.item()) == 0


def test_gradient_of_the_permutation():
    """With weights of one the combine of gradient rows is the gradient of moe_permute's gather."""
    T, d, E, k = 300, 256, 8, 2
    s = M.make_shape(T, d, 128, E, k, capacity=60)
    g = torch.Generator("cuda").manual_seed(1)
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(I32)
    x = torch.randn(T, d, generator=g, device="cuda").to(BF16)
    z = lambda *n: torch.zeros(*n, dtype=I32, device="cuda")
    slot, perm, off, kept = z(T, k), z(T * k), z(E + 1), z(1)
    xp = torch.zeros(T * k, d, dtype=BF16, device="cuda")
    M.moe_permute(s, idx, x, z(E), off, slot, perm, xp, kept, None, M.alloc_workspace(s))
    dxp = torch.randn(T * k, d, generator=g, device="cuda").to(BF16)
    dx = torch.empty_like(x)
    M.moe_combine_rows(s, dxp, slot, None, None, dx)
    n = int(kept.item())
    assert n < T * k                       # some assignments were dropped
    ref = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    ref.index_add_(0, perm[:n].long(), dxp[:n].double())
    mag = torch.zeros_like(ref).index_add_(0, perm[:n].long(), dxp[:n].double().abs())
    assert bool(((dx.double() - ref).abs() <= U * ref.abs() + 4 * 2.0 ** -24 * mag).all())


def test_slots_past_the_rows_are_flagged():
    T, d, k = 4, 128, 2
    s = M.make_shape(T, d, 128, 8, k)
    slot, y, w, R, _ = make(T, d, k, 0.0)
    good = slot.clone()
    slot[2, 1] = T * k
    status = torch.zeros(1, dtype=I32, device="cuda")
    out = torch.empty(T, d, dtype=BF16, device="cuda")
    M.moe_combine_rows(s, y, slot, w, R, out, status)
    assert int(status.item()) == 1 << M.MOE_ERR_CHECK
    good[2, 1] = -1
    ref = torch.empty_like(out)
    M.moe_combine_rows(s, y, good, w, R, ref, None)
    assert torch.equal(out, ref)
    status.zero_()
    dw = torch.full((T, k), 5.0, device="cuda")
    M.moe_combine_rows_backward(s, R, y, slot, w, torch.zeros_like(y), dw, status)
    assert int(status.item()) == 1 << M.MOE_ERR_CHECK and float(dw[2, 1]) == 0.0


def test_stream_and_graph():
    T, d, k = 50, 512, 4
    s = M.make_shape(T, d, 128, 8, k)
    slot, y, w, R, _ = make(T, d, k, 0.2)
    ref = torch.empty(T, d, dtype=BF16, device="cuda")
    M.moe_combine_rows(s, y, slot, w, R, ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.zeros_like(ref)
    side.wait_stream(torch.cuda.current_stream())
    M.moe_combine_rows(s, y, slot, w, R, out, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.moe_combine_rows(s, y, slot, w, R, out)
        M.moe_combine_rows_backward(s, R, y, slot, w, dy, dw)
    w.mul_(0.5)
    g.replay()
    M.moe_combine_rows(s, y, slot, w, R, ref)
    dy2, dw2 = torch.zeros_like(y), torch.zeros_like(w)
    M.moe_combine_rows_backward(s, R, y, slot, w, dy2, dw2)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(dy, dy2) and torch.equal(dw, dw2)
