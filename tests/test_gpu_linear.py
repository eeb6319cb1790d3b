"""The linear products (dense and grouped by expert) and their gradients against
the definition in fp64, at the sizes and groups where they can go wrong.

Bounds, elementwise. u = 2^-8 is half a step of bf16 relative to the value. A
product of two bf16 values is exact in fp32; the tensor cores add 16 products
at a time to an accumulator whose bits below fp32's are cut off, so a sum of K
products is off by at most (K / 16 + 16) 2^-22 S, S the sum of the products'
magnitudes (a factor 2 of room). The activations' fp32 formulas are off by less
than 2^-18 (1 + |z|) and have slopes below 1.13.
"""
import math

import pytest
import torch

from sparse_mixture_experts_17_b200 import moe as M

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
ACTS = {"none": M.MOE_ACT_NONE, "relu": M.MOE_ACT_RELU, "gelu": M.MOE_ACT_GELU,
        "gelu_tanh": M.MOE_ACT_GELU_TANH, "silu": M.MOE_ACT_SILU}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_17_b200 import build
    build.build()


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    z = z.clone().requires_grad_(True)
    (d,) = torch.autograd.grad(act64(z, act).sum(), z)
    if act == "relu":
        d = (z > 0).double()
    return d.detach()


def acc_bound(K, S):
    return (K / 16 + 16) * 2.0 ** -22 * S


def assert_within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), \
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - bound).max()):.3e} over, " \
        f"first at {bad.nonzero()[0].tolist()}"


def rand(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def sizes_to_offsets(sizes, first=0):
    o = [first]
    for n in sizes:
        o.append(o[-1] + n)
    return o


class Case:
    """Inputs of one product; rows outside the groups hold NaN."""

    def __init__(self, rows, di, do, act, offsets=None, seed=0, bias=True):
        g = torch.Generator("cuda").manual_seed(seed)
        self.rows, self.di, self.do, self.act = rows, di, do, act
        self.E = 1 if offsets is None else len(offsets) - 1
        self.b = [0, rows] if offsets is None else offsets
        self.offsets = None if offsets is None else torch.tensor(offsets, dtype=I32, device="cuda")
        self.x = rand(g, rows, di)
        self.W = rand(g, self.E, do, di, std=0.5 / math.sqrt(di) + 0.02)
        self.bias = rand(g, self.E, do, std=0.3, dtype=F32) if bias else None
        self.R = rand(g, rows, do)
        self.dy = rand(g, rows, do)
        self.z = rand(g, rows, do) if act != "none" else None
        self.inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
        self.inside[self.b[0]:self.b[-1]] = True
        for t in (self.x, self.dy, self.R) + ((self.z,) if self.z is not None else ()):
            t[~self.inside] = float("nan")
        self.shape = M.make_linear(rows, di, do, E=self.E, act=ACTS[act])
        self.status = torch.zeros(1, dtype=I32, device="cuda")

    def groups(self):
        return [(e, slice(self.b[e], self.b[e + 1])) for e in range(self.E) if self.b[e + 1] > self.b[e]]

    def forward(self, residual=True, save_z=True, y=None):
        y = torch.full((self.rows, self.do), 7.0, dtype=BF16, device="cuda") if y is None else y
        z = torch.full_like(y, -3.0) if save_z else None
        M.moe_linear_forward(self.shape, self.x, self.offsets, self.W, self.bias,
                             self.R if residual else None, y, z, self.status)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        return y, z

    def check_forward(self, y, z, residual=True):
        for e, r in self.groups():
            x, W = self.x[r].double(), self.W[e].double()
            zr, S = x @ W.T, x.abs() @ W.abs().T
            if self.bias is not None:
                zr, S = zr + self.bias[e].double(), S + self.bias[e].double().abs()
            acc = acc_bound(self.di, S)
            if z is not None:
                assert_within(z[r], zr, U * zr.abs() + (1 + U) * acc, f"z of group {e}")
            ref = act64(zr, self.act)
            if residual:
                ref = ref + self.R[r].double()
            pre = 1.13 * acc + 2.0 ** -18 * (1 + zr.abs())
            assert_within(y[r], ref, U * ref.abs() + (1 + U) * pre, f"y of group {e}")
        out = ~self.inside
        assert bool((y[out] == 7.0).all()) and (z is None or bool((z[out] == -3.0).all()))

    def backward(self, dx=True, dW=True, db=True, ws=None):
        o = dict(dx=torch.full((self.rows, self.di), 5.0, dtype=BF16, device="cuda") if dx else None,
                 dW=torch.full((self.E, self.do, self.di), 5.0, dtype=BF16, device="cuda") if dW else None,
                 db=torch.full((self.E, self.do), 5.0, dtype=F32, device="cuda") if db else None)
        ws = M.alloc_linear_workspace(self.shape) if ws is None else ws
        M.moe_linear_backward(self.shape, self.x, self.offsets, self.W, self.z, self.dy, o["dx"],
                              o["dW"], o["db"], self.status, ws)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        return o

    def check_backward(self, o):
        done = set()
        for e, r in self.groups():
            done.add(e)
            n = r.stop - r.start
            dz = self.dy[r].double()
            ez = torch.zeros_like(dz)          # error of dz before its rounding
            if self.z is not None:
                zz = self.z[r].double()
                ez = 2.0 ** -18 * (1 + zz.abs()) * dz.abs()
                dz = dz * slope64(zz, self.act)
            if o["db"] is not None:
                assert_within(o["db"][e], dz.sum(0), (ez + n * 2.0 ** -24 * dz.abs()).sum(0) + 1e-30,
                              f"db of group {e}")
            er = ez + (U * (dz.abs() + ez) if self.z is not None else 0)   # and after it
            W, x = self.W[e].double(), self.x[r].double()
            if o["dx"] is not None:
                ref = dz @ W
                pre = er @ W.abs() + acc_bound(self.do, (dz.abs() + er) @ W.abs())
                assert_within(o["dx"][r], ref, U * ref.abs() + (1 + U) * pre, f"dx of group {e}")
            if o["dW"] is not None:
                ref = dz.T @ x
                pre = er.T @ x.abs() + acc_bound(n, (dz.abs() + er).T @ x.abs())
                assert_within(o["dW"][e], ref, U * ref.abs() + (1 + U) * pre, f"dW of group {e}")
        for e in set(range(self.E)) - done:
            assert o["dW"] is None or bool((o["dW"][e] == 0).all()), f"dW of empty group {e}"
            assert o["db"] is None or bool((o["db"][e] == 0).all()), f"db of empty group {e}"
        assert o["dx"] is None or bool((o["dx"][~self.inside] == 5.0).all())


DENSE = [(1, 8, 8), (1, 64, 128), (1, 1024, 264), (2, 72, 40), (3, 200, 520), (16, 512, 136), (17, 128, 128),
         (31, 136, 248), (33, 648, 72), (64, 64, 64), (65, 320, 200), (100, 256, 384), (127, 1000, 88),
         (128, 128, 256), (129, 192, 640), (255, 72, 1032), (257, 584, 328), (300, 2048, 96),
         (513, 96, 2056), (1000, 776, 512), (2049, 264, 264), (5000, 136, 264)]


@pytest.mark.parametrize("rows,di,do", DENSE)
def test_dense_forward(rows, di, do):
    act = list(ACTS)[(rows + di) % 5]
    c = Case(rows, di, do, act, seed=rows)
    c.check_forward(*c.forward())


@pytest.mark.parametrize("rows,di,do", DENSE)
def test_dense_backward(rows, di, do):
    act = list(ACTS)[(rows + do) % 5]
    c = Case(rows, di, do, act, seed=rows + 1)
    c.check_backward(c.backward())


GROUPS = {
    "empty_first_last": (200, sizes_to_offsets([0, 0, 70, 0, 63, 1, 66, 0])),
    "one_row_each": (9, sizes_to_offsets([1] * 9)),
    "all_in_one": (500, sizes_to_offsets([0, 0, 500, 0])),
    "all_empty": (64, sizes_to_offsets([0] * 5)),
    "tail_rows": (400, sizes_to_offsets([33, 0, 129, 64, 5])),
    "late_start": (300, sizes_to_offsets([65, 31, 100], first=17)),
    "skewed": (1500, sizes_to_offsets([1, 700, 2, 0, 300, 17, 255, 129, 64, 3])),
    "two_tokens": (4, sizes_to_offsets([0, 1, 0, 0, 2, 0, 1, 0])),
    "many": (1024, sizes_to_offsets([(7 * i) % 9 for i in range(250)])),
    "max_groups": (600, sizes_to_offsets([(i % 5 == 0) * 11 for i in range(256)])),
    "one_group": (77, sizes_to_offsets([77])),
}


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("di,do", [(64, 64), (200, 136), (520, 776)])
def test_grouped_forward(name, di, do):
    rows, off = GROUPS[name]
    c = Case(rows, di, do, list(ACTS)[(rows + di) % 5], offsets=off, seed=rows)
    c.check_forward(*c.forward())


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("di,do", [(64, 64), (200, 136), (520, 776)])
def test_grouped_backward(name, di, do):
    rows, off = GROUPS[name]
    c = Case(rows, di, do, list(ACTS)[(rows + di + 1) % 5], offsets=off, seed=rows)
    c.check_backward(c.backward())


@pytest.mark.parametrize("rows,di,do,off", [
    (8192, 1032, 1288, None), (16384, 520, 256, None), (700, 4096, 1024, None), (6000, 512, 1024, "16"),
    (40, 4096, 2048, "8"), (12000, 264, 520, "200"), (1, 14336, 512, None), (8, 8192, 4096, None)])
def test_larger(rows, di, do, off):
    offsets = None
    if off:
        g = torch.Generator().manual_seed(rows)
        cut = torch.randint(0, rows + 1, (int(off) - 1,), generator=g).sort().values.tolist()
        offsets = [0] + cut + [rows]
    c = Case(rows, di, do, "gelu_tanh", offsets=offsets, seed=rows)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [5, 300])
def test_activations(act, rows):
    """Every activation at small and large |z| (the bias carries z from -60 to 60)."""
    c = Case(rows, 64, 256, act, seed=3)
    c.bias = torch.linspace(-60, 60, 256, device="cuda")[None].contiguous()
    c.check_forward(*c.forward(residual=False), residual=False)
    if c.z is not None:
        c.z = (torch.linspace(-60, 60, 256, device="cuda") +
               0.1 * torch.randn(rows, 256, device="cuda")).to(BF16)
    c.check_backward(c.backward())


def test_optional_arguments():
    rows, off = GROUPS["tail_rows"]
    c = Case(rows, 128, 192, "silu", offsets=off, bias=False)
    y, _ = c.forward(residual=False, save_z=False)
    c.check_forward(y, None, residual=False)
    full = c.backward()
    for kw in (dict(dx=False, dW=False), dict(dx=False, db=False), dict(dW=False, db=False), dict(db=False)):
        part = c.backward(**kw)
        for k, v in part.items():
            assert v is None or torch.equal(v, full[k]), (kw, k)


@pytest.mark.parametrize("rows", [3, 400])
def test_residual_in_place(rows):
    c = Case(rows, 128, 264, "relu")
    y, _ = c.forward(save_z=False)
    z = c.R.clone()
    M.moe_linear_forward(c.shape, c.x, None, c.W, c.bias, z, z, None, c.status)
    torch.cuda.synchronize()
    assert torch.equal(z, y)


@pytest.mark.parametrize("bad", [torch.inf, -torch.inf, torch.nan])
@pytest.mark.parametrize("sizes", [[3, 60, 1], [300, 200, 70]])
def test_non_finite_values_stay_in_their_rows_and_groups(bad, sizes):
    """Infinities and NaN in one group's x, W and dy reach that group's results only."""
    off = sizes_to_offsets(sizes)
    c = Case(off[-1], 136, 200, "none", offsets=off, bias=True)
    ref_y, _ = c.forward(save_z=False)
    ref = c.backward()
    r = off[1]
    c.x[r, 5] = bad          # first row of group 1
    c.dy[off[2] - 1, 7] = bad    # its last row
    c.W[1, 3, 2] = bad
    y, _ = c.forward(save_z=False)
    o = c.backward()
    keep = torch.ones(off[-1], dtype=torch.bool, device="cuda")
    keep[off[1]:off[2]] = False
    assert torch.equal(y[keep], ref_y[keep])
    assert torch.equal(o["dx"][keep], ref["dx"][keep])
    for e in (0, 2):
        assert torch.equal(o["dW"][e], ref["dW"][e]) and torch.equal(o["db"][e], ref["db"][e])
    assert not bool(torch.isfinite(y[r].float()).any())       # the whole row: x[r, 5] meets every W row
    others = slice(off[1] + 1, off[2])
    if sizes[1] > 1:
        assert not bool(torch.isfinite(y[others, 3].float()).any())
        assert bool(torch.isfinite(y[others, 4:].float()).all())


@pytest.mark.parametrize("offsets", [[0, 50, 40, 100], [-1, 20, 40, 100], [0, 20, 40, 101],
                                     [5, 3, 2, 1], [0, 100, 0, 100], [0, 2 ** 31 - 1, 10, 100]])
def test_broken_offsets_are_flagged(offsets):
    """Decreasing or outside [0, rows]: flagged, every group empty, nothing else written."""
    for rows in (100,):
        c = Case(rows, 64, 72, "relu", offsets=[0, 20, 40, 100])
        c.offsets = torch.tensor(offsets, dtype=I32, device="cuda")
        y = torch.full((rows, 72), 7.0, dtype=BF16, device="cuda")
        M.moe_linear_forward(c.shape, c.x, c.offsets, c.W, c.bias, c.R, y, None, c.status)
        torch.cuda.synchronize()
        assert int(c.status.item()) == 1 << M.MOE_ERR_CHECK
        assert bool((y == 7.0).all())
        c.status.zero_()
        dx = torch.full((rows, 64), 5.0, dtype=BF16, device="cuda")
        dW = torch.full((3, 72, 64), 5.0, dtype=BF16, device="cuda")
        db = torch.full((3, 72), 5.0, dtype=F32, device="cuda")
        M.moe_linear_backward(c.shape, c.x, c.offsets, c.W, c.z, c.dy, dx, dW, db, c.status,
                              M.alloc_linear_workspace(c.shape))
        torch.cuda.synchronize()
        assert int(c.status.item()) == 1 << M.MOE_ERR_CHECK
        assert bool((dx == 5.0).all()) and bool((dW == 0).all()) and bool((db == 0).all())


def test_no_rows():
    s = M.make_linear(0, 64, 72, E=3)
    off = torch.zeros(4, dtype=I32, device="cuda")
    dW = torch.full((3, 72, 64), 5.0, dtype=BF16, device="cuda")
    db = torch.full((3, 72), 5.0, dtype=F32, device="cuda")
    x = torch.zeros(0, 64, dtype=BF16, device="cuda")
    y = torch.zeros(0, 72, dtype=BF16, device="cuda")
    M.moe_linear_forward(s, x, off, torch.zeros(3, 72, 64, dtype=BF16, device="cuda"), None, None, y)
    M.moe_linear_backward(s, x, off, None, None, y, None, dW, db, None, None)
    torch.cuda.synchronize()
    assert bool((dW == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("rows,di,do,off", [(2, 512, 1024, None), (300, 520, 264, None),
                                            (3000, 264, 328, sizes_to_offsets([1500, 0, 100, 1400]))])
def test_repeats_bit_for_bit(rows, di, do, off):
    c = Case(rows, di, do, "gelu", offsets=off)
    y0, z0 = c.forward()
    o0 = c.backward()
    ws = M.alloc_linear_workspace(c.shape).fill_(255)       # NaN patterns: nothing is read before it is written
    for _ in range(3):
        y, z = c.forward()
        o = c.backward(ws=ws)
        assert torch.equal(y[c.inside], y0[c.inside]) and torch.equal(z[c.inside], z0[c.inside])
        for k in o:
            assert torch.equal(o[k], o0[k]), k


@pytest.mark.parametrize("rows,off", [(2, None), (700, sizes_to_offsets([300, 0, 333, 67]))])
def test_other_stream_and_captured_graphs(rows, off):
    """Eager on another stream; then two captured graphs over the same workspace, replayed on
    new inputs in turn, follow the inputs (and the offsets) of the moment."""
    c = Case(rows, 264, 520, "silu", offsets=off)
    y_ref, z_ref = c.forward()
    o_ref = c.backward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.full_like(y_ref, 7.0)
    M.moe_linear_forward(c.shape, c.x, c.offsets, c.W, c.bias, c.R, y, None, c.status, stream=side)
    side.synchronize()
    assert torch.equal(y, y_ref)
    ws = M.alloc_linear_workspace(c.shape)
    outs = [dict(y=torch.zeros_like(y_ref), z=torch.zeros_like(y_ref), dx=torch.zeros_like(c.x),
                 dW=torch.zeros_like(c.W), db=torch.zeros_like(o_ref["db"])) for _ in range(2)]

    def both(o):
        M.moe_linear_forward(c.shape, c.x, c.offsets, c.W, c.bias, c.R, o["y"], o["z"], c.status)
        M.moe_linear_backward(c.shape, c.x, c.offsets, c.W, c.z, c.dy, o["dx"], o["dW"], o["db"],
                              c.status, ws)
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both(o)
        graphs.append(g)
    for trial in range(2):
        if trial:                        # new values, and other groups
            c.x.copy_(torch.flip(c.x, (0,)))
            c.dy.mul_(2)
            if off:
                c.b = sizes_to_offsets([0, 650, 1, 49])
                c.offsets.copy_(torch.tensor(c.b, dtype=I32))
        for g, o in zip(graphs, outs):
            for v in o.values():
                v.fill_(5.0)
            o["y"].fill_(7.0)
            o["z"].fill_(-3.0)
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            c.check_forward(o["y"], o["z"])
            c.check_backward({k: o[k] for k in ("dx", "dW", "db")})


def test_gradient_against_differences():
    """The analytic gradient of sum(y dy) against central differences of the fp64 definition
    (the chain the kernels are tested against above)."""
    for act in ACTS:
        z = torch.linspace(-4, 4, 81, dtype=F64) + 0.013
        h = 1e-5
        diff = (act64(z + h, act) - act64(z - h, act)) / (2 * h)
        assert float((diff - slope64(z, act)).abs().max()) < 1e-8, act
    # and the kernels' dx along a direction: y(x + h v) - y(x - h v) over 2 h, in fp64 from dx and W
    c = Case(48, 64, 72, "gelu_tanh", seed=9)
    z64 = c.x.double() @ c.W[0].double().T + c.bias[0].double()
    c.z = z64.to(BF16)
    o = c.backward()
    v = torch.randn(48, 64, device="cuda", dtype=F64)
    f = lambda t: (act64((c.x.double() + t * v) @ c.W[0].double().T + c.bias[0].double(), c.act) *
                   c.dy.double()).sum()
    diff = float((f(1e-5) - f(-1e-5)) / 2e-5)
    got = float((o["dx"].double() * v).sum())
    # dx carries its own rounding and those of z and dz: at most 4 U per term
    room = 4 * U * float((c.dy.double().abs() @ c.W[0].double().abs()).mul(v.abs()).sum())
    assert abs(got - diff) <= room
