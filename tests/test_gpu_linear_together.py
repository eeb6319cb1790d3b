"""The linear products, the combine of bf16 rows and the gradient clipping as a layer
uses them together, and the linear products where their tiles and rings change.

A layer of plain experts (no gate): route, permute, up product with gelu, down
product, combine onto the residual stream; then the gradients back through all
of it, clipped together. Every stage is checked against the definition in fp64 on
the inputs that it really got, with the bounds of its own test, and the whole runs
once more as a captured graph, bit for bit the same.
"""
import math

import pytest
import torch

from sparse_mixture_experts_17_b200 import moe as M
from test_gpu_linear import (BF16, F32, F64, I32, U, Case, acc_bound, act64, assert_within, rand,
                             sizes_to_offsets, slope64)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_17_b200 import build
    build.build()


class Layer:
    """Device state of one layer of plain experts and its gradients."""

    def __init__(self, T, d, d_ff, E, k, capacity, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        self.T, self.d, self.d_ff, self.E, self.k = T, d, d_ff, E, k
        n = T * k
        self.shape = M.make_shape(T, d, d_ff, E, k, capacity=capacity)
        self.up = M.make_linear(n, d, d_ff, E=E, act=M.MOE_ACT_GELU)
        self.down = M.make_linear(n, d_ff, d, E=E)
        self.x, self.dout = rand(g, T, d), rand(g, T, d)
        self.Wg = rand(g, E, d, std=0.05)
        self.W1, self.W2 = rand(g, E, d_ff, d, std=1 / math.sqrt(d)), rand(g, E, d, d_ff, std=1 / math.sqrt(d_ff))
        self.b1, self.b2 = rand(g, E, d_ff, std=0.1, dtype=F32), rand(g, E, d, std=0.1, dtype=F32)
        new = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device="cuda")
        self.logits, self.idx, self.w = new(T, E, dtype=F32), new(T, k, dtype=I32), new(T, k, dtype=F32)
        self.counts, self.off, self.kept = new(E, dtype=I32), new(E + 1, dtype=I32), new(1, dtype=I32)
        self.slot, self.perm, self.xp = new(T, k, dtype=I32), new(n, dtype=I32), new(n, d)
        self.z, self.h, self.y, self.out = new(n, d_ff), new(n, d_ff), new(n, d), new(T, d)
        self.dy, self.dw, self.dh, self.dxp = new(n, d), new(T, k, dtype=F32), new(n, d_ff), new(n, d)
        self.dW1, self.dW2 = torch.zeros_like(self.W1), torch.zeros_like(self.W2)
        self.db1, self.db2, self.dx = torch.zeros_like(self.b1), torch.zeros_like(self.b2), new(T, d)
        self.grads = [self.dW1, self.dW2, self.db1, self.db2]
        self.clipped = [torch.zeros_like(t) for t in self.grads]
        self.norm, self.status = new(1, dtype=F32), new(1, dtype=I32)
        self.ws = M.alloc_workspace(self.shape)
        self.ws1, self.ws2 = M.alloc_linear_workspace(self.up), M.alloc_linear_workspace(self.down)
        self.gws = M.alloc_grad_workspace(self.grads)

    def run(self, max_norm):
        M.moe_route(self.shape, self.x, self.Wg, None, self.logits, self.idx, self.w, self.status, self.ws)
        M.moe_permute(self.shape, self.idx, self.x, self.counts, self.off, self.slot, self.perm, self.xp,
                      self.kept, self.status, self.ws)
        M.moe_linear_forward(self.up, self.xp, self.off, self.W1, self.b1, None, self.h, self.z, self.status)
        M.moe_linear_forward(self.down, self.h, self.off, self.W2, self.b2, None, self.y, None, self.status)
        M.moe_combine_rows(self.shape, self.y, self.slot, self.w, self.x, self.out, self.status)
        M.moe_combine_rows_backward(self.shape, self.dout, self.y, self.slot, self.w, self.dy, self.dw, self.status)
        M.moe_linear_backward(self.down, self.h, self.off, self.W2, None, self.dy, self.dh, self.dW2, self.db2,
                              self.status, self.ws2)
        M.moe_linear_backward(self.up, self.xp, self.off, self.W1, self.z, self.dh, self.dxp, self.dW1, self.db1,
                              self.status, self.ws1)
        # the gather's gradient, and the residual's
        M.moe_combine_rows(self.shape, self.dxp, self.slot, None, self.dout, self.dx, self.status)
        M.moe_clip_grads(self.grads, max_norm, self.norm, self.clipped, self.status, self.gws)

    def outputs(self):
        return dict(out=self.out, dw=self.dw, dx=self.dx, dW1=self.dW1, dW2=self.dW2, db1=self.db1,
                    db2=self.db2, norm=self.norm, **{f"clipped{i}": t for i, t in enumerate(self.clipped)})


def _check_product(x, W, bias, act, off, y, z):
    for e in range(W.shape[0]):
        r = slice(off[e], off[e + 1])
        xr, We = x[r].double(), W[e].double()
        zr = xr @ We.T + bias[e].double()
        acc = acc_bound(W.shape[2], xr.abs() @ We.abs().T + bias[e].double().abs())
        if z is not None:
            assert_within(z[r], zr, U * zr.abs() + (1 + U) * acc, f"z of group {e}")
        ref = act64(zr, act)
        assert_within(y[r], ref, U * ref.abs() + (1 + U) * (1.13 * acc + 2.0 ** -18 * (1 + zr.abs())), f"y of group {e}")


def _check_gradients(x, W, z, act, off, dy, dx, dW, db):
    for e in range(W.shape[0]):
        r = slice(off[e], off[e + 1])
        n = r.stop - r.start
        dz = dy[r].double()
        ez = torch.zeros_like(dz)
        er = ez
        if z is not None:
            zz = z[r].double()
            ez = 2.0 ** -18 * (1 + zz.abs()) * dz.abs()
            dz = dz * slope64(zz, act)
            er = ez + U * (dz.abs() + ez)
        assert_within(db[e], dz.sum(0), (ez + n * 2.0 ** -24 * dz.abs()).sum(0) + 1e-30, f"db of group {e}")
        xr, We = x[r].double(), W[e].double()
        ref = dz @ We
        assert_within(dx[r], ref, U * ref.abs() + (1 + U) * (er @ We.abs() + acc_bound(W.shape[1], (dz.abs() + er) @ We.abs())),
                      f"dx of group {e}")
        ref = dz.T @ xr
        assert_within(dW[e], ref, U * ref.abs() + (1 + U) * (er.T @ xr.abs() + acc_bound(n, (dz.abs() + er).T @ xr.abs())),
                      f"dW of group {e}")


@pytest.mark.parametrize("T,d,d_ff,E,k,capacity", [
    (1, 256, 384, 8, 2, 0), (37, 128, 256, 8, 2, 0), (300, 256, 384, 16, 4, 60), (2048, 512, 768, 8, 2, 0)])
def test_layer_of_plain_experts(T, d, d_ff, E, k, capacity):
    L = Layer(T, d, d_ff, E, k, capacity, seed=T)
    L.run(max_norm=0.5)
    torch.cuda.synchronize()
    assert int(L.status.item()) == 0
    off = L.off.tolist()
    slot = L.slot.long()
    kept = slot >= 0
    assert off[-1] == int(kept.sum()) and (capacity or off[-1] == T * k)
    assert torch.equal(L.xp[slot[kept]], L.x[kept.nonzero()[:, 0]])
    _check_product(L.xp, L.W1, L.b1, "gelu", off, L.h, L.z)
    _check_product(L.h, L.W2, L.b2, "none", off, L.y, None)
    rows = torch.cat([L.y.double(), torch.zeros(1, d, dtype=F64, device="cuda")])[slot]      # slot -1: the zero row
    w = L.w.double().unsqueeze(-1)
    ref, S = L.x.double() + (w * rows).sum(1), L.x.double().abs() + (w * rows).abs().sum(1)
    assert_within(L.out, ref, U * ref.abs() + (k + 1) * 2.0 ** -23 * S, "out")
    # backward
    dot = (L.dout.double().unsqueeze(1) * rows).sum(-1)
    bound = d * 2.0 ** -24 * (L.dout.double().unsqueeze(1) * rows).abs().sum(-1) + 1e-30
    assert_within(L.dw, dot, bound, "dw")
    dy_ref = (w * L.dout.double().unsqueeze(1))[kept]
    assert_within(L.dy[slot[kept]], dy_ref, (U + 2.0 ** -23) * dy_ref.abs(), "dy")
    _check_gradients(L.h, L.W2, None, "none", off, L.dy, L.dh, L.dW2, L.db2)
    _check_gradients(L.xp, L.W1, L.z, "gelu", off, L.dh, L.dxp, L.dW1, L.db1)
    rows = torch.cat([L.dxp.double(), torch.zeros(1, d, dtype=F64, device="cuda")])[slot]
    ref, S = L.dout.double() + rows.sum(1), L.dout.double().abs() + rows.abs().sum(1)
    assert_within(L.dx, ref, U * ref.abs() + (k + 1) * 2.0 ** -23 * S, "dx")
    norm = math.sqrt(sum(float((t.double() ** 2).sum()) for t in L.grads))
    assert abs(float(L.norm) - norm) <= 2.0 ** -18 * norm
    c = min(1.0, 0.5 / (norm + 1e-6))
    for got, g in zip(L.clipped, L.grads):
        ref = c * g.double()
        u = U if g.dtype == BF16 else 2.0 ** -24
        assert_within(got, ref, (u + 2.0 ** -17) * ref.abs() + 1e-38, "clipped")
    # the same as one graph, replayed over poisoned buffers
    first = {n: t.clone() for n, t in L.outputs().items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.run(max_norm=0.5)
    for t in (L.h, L.z, L.y, L.dy, L.dh, L.dxp, L.ws1, L.ws2, *L.outputs().values()):
        t.fill_(3)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert int(L.status.item()) == 0
    for n, t in L.outputs().items():
        assert torch.equal(t, first[n]), n


MIXED = {
    # long groups beside short ones: rings of every class, from both ends
    "mixed": (2048, 256, sizes_to_offsets([600, 5, 40, 70, 0, 100, 300, 129, 64, 65, 1, 250])),
    "short": (2048, 200, sizes_to_offsets([100, 33, 64, 128, 127, 66, 65, 1, 0, 90, 44, 120])),
    # double tiles: even and odd numbers of them, a single last one, and short groups between
    "double": (2048, 4096, sizes_to_offsets([1300, 900, 513, 1030, 257, 70])),
    "double_long": (1032, 4160, sizes_to_offsets([0, 2049, 5, 1500, 3000, 512])),
}


@pytest.mark.parametrize("name", MIXED)
def test_tiles_of_every_class(name):
    do, di, off = MIXED[name]
    rows = off[-1] + 7
    c = Case(rows, di, do, "gelu", offsets=off, seed=5)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())
    # and the same contraction lengths in dx
    c = Case(rows, do, di, "silu", offsets=off, seed=6)
    c.check_backward(c.backward())


@pytest.mark.parametrize("rows,di,do", [(1500, 4160, 4096), (4096, 4096, 2048)])
def test_dense_double_tiles(rows, di, do):
    c = Case(rows, di, do, "gelu_tanh", seed=7)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("rows,di,do,off", [(2048, 512, 1024, None), (90, 256, 512, None),
                                            (1600, 256, 512, sizes_to_offsets([900, 0, 33, 600, 67]))])
def test_outputs_left_out(act, rows, di, do, off):
    """Each output alone and in pairs equals what the whole call gives: the kernels of one call run
    beside each other and wait for what they need."""
    c = Case(rows, di, do, act, offsets=off, seed=11)
    full = c.backward()
    c.check_backward(full)
    for mask in range(1, 7):
        part = c.backward(dx=bool(mask & 1), dW=bool(mask & 2), db=bool(mask & 4))
        for k, v in part.items():
            assert v is None or torch.equal(v, full[k]), (mask, k)


def test_calls_in_a_row():
    """Forward and backward calls of several shapes on one stream, with no wait between them and one
    workspace, give what each gives alone: a call's kernels start while the one before ends."""
    cases = [Case(300, 520, 264, "gelu", seed=1), Case(2, 1024, 4096, "silu", seed=2),
             Case(3000, 264, 328, "relu", offsets=sizes_to_offsets([1500, 0, 100, 1400]), seed=3),
             Case(4096, 256, 2048, "gelu_tanh", seed=4)]
    alone = [(c.forward()[0], c.backward()) for c in cases]
    ws = torch.empty(max(M.moe_linear_workspace_size(c.shape) for c in cases), dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(3):
        for c in cases:
            y = torch.full((c.rows, c.do), 7.0, dtype=BF16, device="cuda")
            dx, dW = torch.full_like(c.x, 5.0), torch.empty_like(c.W)
            db = torch.empty_like(c.bias)
            M.moe_linear_forward(c.shape, c.x, c.offsets, c.W, c.bias, c.R, y, None, c.status)
            M.moe_linear_backward(c.shape, c.x, c.offsets, c.W, c.z, c.dy, dx, dW, db, c.status, ws)
            got.append((y, dict(dx=dx, dW=dW, db=db)))
    torch.cuda.synchronize()
    for i, (y, o) in enumerate(got):
        y0, o0 = alone[i % len(cases)]
        assert torch.equal(y, y0), i
        for k in o:
            assert torch.equal(o[k], o0[k]), (i, k)


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, in flight together give what each gives alone."""
    cases = [Case(900, 520, 2048, "gelu", offsets=sizes_to_offsets([600, 0, 250, 50]), seed=21),
             Case(2100, 1024, 1032, "silu", seed=22)]
    alone = [(c.forward()[0], c.backward()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [M.alloc_linear_workspace(c.shape) for c in cases]
    got = [[(torch.full((c.rows, c.do), 7.0, dtype=BF16, device="cuda"),
             dict(dx=torch.full_like(c.x, 5.0), dW=torch.empty_like(c.W), db=torch.empty_like(c.bias)))
            for _ in range(8)] for c in cases]
    torch.cuda.synchronize()
    for n in range(8):
        for c, st, w, out in zip(cases, streams, ws, got):
            y, o = out[n]
            M.moe_linear_forward(c.shape, c.x, c.offsets, c.W, c.bias, c.R, y, None, c.status, stream=st)
            M.moe_linear_backward(c.shape, c.x, c.offsets, c.W, c.z, c.dy, o["dx"], o["dW"], o["db"], c.status, w,
                                  stream=st)
    torch.cuda.synchronize()
    for (y0, o0), out, c in zip(alone, got, cases):
        assert int(c.status.item()) == 0
        for y, o in out:
            assert torch.equal(y, y0)
            for k in o:
                assert torch.equal(o[k], o0[k]), k


def test_dx_feeds_the_next_call_at_once():
    """A chain of products, each backward fed by the one before without a wait, equals the same with
    waits: the last kernel of a call ends after all others of it."""
    g = torch.Generator("cuda").manual_seed(3)
    n, d = 700, 512
    W = [rand(g, 1, d, d, std=1 / math.sqrt(d)) for _ in range(6)]
    x, dy = rand(g, n, d), rand(g, n, d)
    z = rand(g, n, d)
    s = M.make_linear(n, d, d, act=M.MOE_ACT_SILU)
    ws = M.alloc_linear_workspace(s)

    def chain(wait):
        cur, out = dy, []
        for w in W:
            dx, dW = torch.empty_like(x), torch.empty_like(w)
            db = torch.empty(1, d, dtype=F32, device="cuda")
            M.moe_linear_backward(s, x, None, w, z, cur, dx, dW, db, None, ws)
            if wait:
                torch.cuda.synchronize()
            out += [dx, dW, db]
            cur = dx
        torch.cuda.synchronize()
        return out
    ref = chain(True)
    for _ in range(3):
        for a, b in zip(chain(False), ref):
            assert torch.equal(a, b)


def test_lower_tail_of_gelu():
    """gelu(z) for z from -6 to 0 keeps its relative accuracy, though 1 + erf(z / sqrt 2) cancels there:
    Phi to 6e-6, and one rounding to bf16."""
    z = torch.linspace(-6, 0, 769, device="cuda")[:768].to(BF16)
    W = torch.zeros(768, 8, dtype=BF16, device="cuda")
    W[:, 0] = z
    x = torch.zeros(3, 8, dtype=BF16, device="cuda")
    x[:, 0] = 1.0
    y = torch.empty(3, 768, dtype=BF16, device="cuda")
    M.moe_linear_forward(M.make_linear(3, 8, 768, act=M.MOE_ACT_GELU), x, None, W, None, None, y)
    ref = (z.double() * torch.special.ndtr(z.double())).expand(3, -1)
    assert_within(y, ref, (U + 2.0 ** -17) * ref.abs(), "gelu")


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_bias_gradients_keep_fp32(act):
    """dbias sums the unrounded dz in fp32, so the derivative has to be good to fp32 as well. The special
    functions are off by 2 units in the last place (2.4e-7), their arguments by one rounding each, Phi
    by 1.4e-7 of itself; multiplied by slopes of at most 1.13 and by |z|: below 7e-7 (1 + |z|) in all.
    The sum of n terms adds n 2^-24."""
    c = Case(2190, 64, 616, act, seed=4)
    o = c.backward(dx=False, dW=False)
    dz = c.dy.double() * slope64(c.z.double(), act)
    bound = (7e-7 * (1 + c.z.double().abs()) * c.dy.double().abs() + c.rows * 2.0 ** -24 * dz.abs()).sum(0)
    # and of the whole vector: dy has both signs, independent of z, so the terms' errors, at most 7e-7 of
    # a term where |z| is small and less of it elsewhere, add up as the terms do
    err = o["db"][0].double() - dz.sum(0)
    assert bool((err.abs() <= bound).all())
    assert float(err.norm() / dz.sum(0).norm()) <= 7e-7


@pytest.mark.parametrize("di,do", [(64, 8192), (8192, 64)])
def test_indices_past_32_bits(di, do):
    """2.6 * 2^30 elements in y (or x, and then in dx)."""
    rows = 340000
    g = torch.Generator("cuda").manual_seed(1)
    W = rand(g, 1, do, di, std=1 / math.sqrt(di))
    x = torch.empty(rows, di, dtype=BF16, device="cuda")
    for part in x.split(1 << 15):
        part.copy_(rand(g, *part.shape))
    s = M.make_linear(rows, di, do)
    y = torch.empty(rows, do, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    M.moe_linear_forward(s, x, None, W, None, None, y, None, status)
    dx = torch.empty_like(x)
    M.moe_linear_backward(s, x, None, W, None, y, dx, None, None, status, M.alloc_linear_workspace(s))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for r in (0, 1, rows // 2 + 3, (1 << 31) // max(di, do) - 1, (1 << 31) // max(di, do) + 1, rows - 1):
        xr, W64 = x[r:r + 1].double(), W[0].double()
        ref = xr @ W64.T
        assert_within(y[r:r + 1], ref, U * ref.abs() + (1 + U) * acc_bound(di, xr.abs() @ W64.abs().T), f"y row {r}")
        yr = y[r:r + 1].double()
        ref = yr @ W64
        assert_within(dx[r:r + 1], ref, U * ref.abs() + (1 + U) * acc_bound(do, yr.abs() @ W64.abs()), f"dx row {r}")
