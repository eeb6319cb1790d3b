"""The global gradient norm and clipping against fp64.

Bounds: squares are added in fp32 over at most 32 elements (32 roundings of
2^-24, halved by the root) and in fp64 beyond, and the norm is rounded once:
(16 + 1) 2^-24. A scaled gradient carries the factor's error (the norm's, one
addition, one division) and one product and rounding: 22 2^-24 in fp32, and
2^-8 for a bf16 gradient."""
import math

import pytest
import torch

from sparse_mixture_experts_17_b200 import moe as M

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NORM_REL = 17 * 2.0 ** -24
HALF = {F32: 22 * 2.0 ** -24, BF16: 2.0 ** -8 + 22 * 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_17_b200 import build
    build.build()


def rand(n, dtype, seed, std=1e-3):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * std).to(dtype)


def norm64(grads):
    return math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))


def state():
    return (torch.zeros(1, device="cuda"), torch.zeros(1, dtype=I32, device="cuda"),
            M.alloc_grad_workspace())


def check_clipped(grads, outs, max_norm, norm):
    ref = norm64(grads)
    assert abs(float(norm) - ref) <= NORM_REL * ref + 1e-45
    c = min(1.0, max_norm / (ref + 1e-6))
    for g, o in zip(grads, outs):
        r = g.double() * c
        if c == 1.0:
            assert torch.equal(g, o)
        else:
            tiny = 2.0 ** -149 if g.dtype == F32 else 2.0 ** -133   # half a step of the smallest values
            assert bool(((o.double() - r).abs() <= HALF[g.dtype] * r.abs() + tiny).all())


SETS = {
    "one_value": [(1, F32)],
    "one_bf16": [(1, BF16)],
    "empty_among": [(0, F32), (5, BF16), (0, BF16), (1000, F32)],
    "odd": [(3, F32), (7, BF16), (8, BF16), (9, BF16), (4097, F32), (65537, BF16), (31, F32)],
    "chunk_edges": [(16384, F32), (16383, F32), (16385, F32), (32768, BF16), (32769, BF16)],
    "many": [(17 * i % 300 + 1, F32 if i % 3 else BF16) for i in range(500)],
    "large": [(5_000_011, F32), (3_000_001, BF16)],
}


@pytest.mark.parametrize("name", SETS)
def test_norm_and_clip(name):
    grads = [rand(n, t, i) for i, (n, t) in enumerate(SETS[name])]
    norm, status, ws = state()
    M.moe_grad_norm(grads, norm, status, ws)
    ref = norm64(grads)
    assert abs(float(norm) - ref) <= NORM_REL * ref
    for ratio in (0.5, 3.0):
        max_norm = ref / ratio
        keep = [g.clone() for g in grads]
        outs = [torch.full_like(g, 9.0) for g in grads]
        M.moe_clip_grads(grads, max_norm, norm, outs, status, ws)
        check_clipped(grads, outs, max_norm, norm)
        assert all(torch.equal(g, k) for g, k in zip(grads, keep))     # out of place: untouched
        mine = [g.clone() for g in grads]
        M.moe_clip_grads(mine, max_norm, norm, None, status, ws)
        assert all(torch.equal(a, b) for a, b in zip(mine, outs))
        mixed = [g.clone() for g in grads]                             # some in place, some not
        mo = [m if i % 2 else torch.full_like(m, 9.0) for i, m in enumerate(mixed)]
        M.moe_clip_grads(mixed, max_norm, norm, mo, status, ws)
        assert all(torch.equal(a, b) for a, b in zip(mo, outs))
    assert int(status.item()) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("a", range(8))
def test_alignment(dtype, a):
    """Slices of a flat buffer at every offset: nothing outside them is read into the norm or written."""
    for b in (0, 1, 3, 8):
        flat = torch.full((40000,), float("nan"), dtype=dtype, device="cuda")
        out = torch.full((40000,), 9.0, dtype=dtype, device="cuda")
        cuts = [(a, 20001), (20001 + a, 20003 + a), (30000 + a, 39000)]
        grads = [flat[i:j] for i, j in cuts]
        for i, g in enumerate(grads):
            g.copy_(rand(g.numel(), dtype, i))
        outs = [out[i + b:j + b] for i, j in cuts]
        norm, status, ws = state()
        ref = norm64(grads)
        M.moe_clip_grads(grads, ref / 2, norm, outs, status, ws)
        check_clipped(grads, outs, ref / 2, norm)
        held = torch.zeros(40000, dtype=torch.bool, device="cuda")
        for i, j in cuts:
            held[i + b:j + b] = True
        assert bool((out[~held] == 9.0).all()) and int(status.item()) == 0


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-10, 1e15, 1e25, 1e30])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_squares_outside_fp32(scale, dtype):
    """Norms whose squares overflow or vanish in fp32."""
    grads = [rand(10007, dtype, 1, std=scale), torch.zeros(5000, dtype=dtype, device="cuda")]
    norm, status, ws = state()
    M.moe_grad_norm(grads, norm, status, ws)
    ref = norm64(grads)
    assert abs(float(norm) - ref) <= NORM_REL * ref and int(status.item()) == 0
    one = torch.zeros(9999, dtype=dtype, device="cuda")     # a single tiny value among zeros
    one[777] = scale
    M.moe_grad_norm([one], norm, status, ws)
    assert abs(float(norm) - float(one[777])) <= NORM_REL * float(one[777])


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [0, 5000, 10006])
def test_non_finite(bad, at):
    g = rand(10007, F32, 2)
    g[at] = bad
    h = rand(33, BF16, 3)
    keep = [g.clone(), h.clone()]
    norm, status, ws = state()
    M.moe_clip_grads([g, h], 1e-3, norm, None, status, ws)
    assert int(status.item()) == 1 << M.MOE_ERR_NONFINITE and not math.isfinite(float(norm))
    outs = [torch.zeros_like(g), torch.zeros_like(h)]
    M.moe_clip_grads([g, h], 1e-3, norm, outs, status, ws)
    for a, b, o in zip(keep, (g, h), outs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(a.view(torch.uint8), o.view(torch.uint8))
    status.zero_()
    M.moe_grad_norm([g, h], norm, status, ws)
    assert int(status.item()) == 1 << M.MOE_ERR_NONFINITE


def test_none_and_zero():
    norm, status, ws = state()
    norm.fill_(5)
    M.moe_grad_norm([], norm, status, ws)
    assert float(norm) == 0.0
    norm.fill_(5)
    M.moe_clip_grads([], 1.0, norm, None, status, ws)
    assert float(norm) == 0.0
    z = torch.zeros(100, device="cuda")
    M.moe_clip_grads([z], 1.0, norm, None, status, ws)
    assert float(norm) == 0.0 and bool((z == 0).all()) and int(status.item()) == 0
    g = rand(100, F32, 1)
    keep = g.clone()
    M.moe_clip_grads([g], math.inf, norm, None, status, ws)     # no limit: the norm alone
    assert torch.equal(g, keep)


def test_views_of_matrices_and_repeats():
    """Tensors of any shape; the same bits on every call, on a used workspace too."""
    grads = [rand(300 * 70, F32, 1).reshape(300, 70), rand(64 * 128, BF16, 2).reshape(2, 32, 128)]
    norm, status, ws = state()
    ws.fill_(255)
    got = set()
    for _ in range(4):
        M.moe_grad_norm(grads, norm, status, ws)
        got.add(float(norm))
    assert len(got) == 1
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_grad_norm([grads[0].T], norm, status, ws)
    with pytest.raises(TypeError, match="float16"):
        M.moe_grad_norm([grads[0].half()], norm, status, ws)
    with pytest.raises(M.MoeError):                              # the same tensor twice
        M.moe_clip_grads([grads[0], grads[0]], 1.0, norm, None, status, ws)
    M.moe_grad_norm([grads[0], grads[0]], norm, status, ws)      # for the norm alone it counts twice
    ref = norm64([grads[0], grads[0]])
    assert abs(float(norm) - ref) <= NORM_REL * ref


def test_stream_and_two_graphs_on_one_workspace():
    grads = [rand(70001, F32, 1), rand(333, BF16, 2)]
    outs = [[torch.zeros_like(g) for g in grads] for _ in range(2)]
    norms = [torch.zeros(1, device="cuda") for _ in range(2)]
    _, status, ws = state()
    limit = [norm64(grads) / 4, norm64(grads) / 2]
    graphs = []
    for o, n, m in zip(outs, norms, limit):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            M.moe_clip_grads(grads, m, n, o, status, ws)
        graphs.append(g)
    for factor in (1.0, 1.7):
        grads[0].mul_(factor)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, n, m in zip(outs, norms, limit):
            check_clipped(grads, o, m, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    M.moe_grad_norm(grads, norms[1], status, ws, stream=side)
    side.synchronize()
    assert float(norms[1]) == float(norms[0])
