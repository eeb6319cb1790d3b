"""The linear products, the combine of bf16 rows and the gradient clipping on a
machine without a GPU: workspace sizes and every refusal happen on the host,
before anything is launched (no call here reaches a device)."""
import ctypes

import pytest
import torch

from sparse_mixture_experts_17_b200 import build as B
from sparse_mixture_experts_17_b200 import moe as M

FAKE = 0x100000     # an aligned non-null address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.lib()


def _fwd(lib, s, x=FAKE, off=FAKE, W=FAKE, bias=None, res=None, y=FAKE, z=None):
    return lib.moe_linear_forward(ctypes.byref(s), x, off, W, bias, res, y, z, None, None)


def _bwd(lib, s, x=FAKE, off=FAKE, W=FAKE, z=FAKE, dy=FAKE, dx=FAKE, dW=FAKE, db=FAKE, ws=FAKE,
         n=1 << 40):
    return lib.moe_linear_backward(ctypes.byref(s), x, off, W, z, dy, dx, dW, db, None, ws, n, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=(1 << 24) + 1), dict(d_in=0), dict(d_in=4), dict(d_in=12),
    dict(d_in=65544), dict(d_out=-8), dict(d_out=20), dict(d_out=65544), dict(E=0), dict(E=257),
    dict(act=-1), dict(act=5), dict(flags=1),
])
def test_bad_shapes(lib, bad):
    kw = dict(rows=64, d_in=128, d_out=256, E=8, act=M.MOE_ACT_RELU) | bad
    s = M.moe_linear_t(kw["rows"], kw["d_in"], kw["d_out"], kw["E"], kw["act"], kw.get("flags", 0))
    n = ctypes.c_size_t(0)
    assert lib.moe_linear_workspace_size(ctypes.byref(s), ctypes.byref(n)) == M.MOE_ERR_INVALID_ARG
    assert _fwd(lib, s) == M.MOE_ERR_INVALID_ARG
    assert _bwd(lib, s) == M.MOE_ERR_INVALID_ARG


def test_linear_refusals(lib):
    s = M.make_linear(64, 128, 256, E=8, act=M.MOE_ACT_GELU)
    assert lib.moe_linear_workspace_size(ctypes.byref(s), None) == M.MOE_ERR_INVALID_ARG
    assert lib.moe_linear_workspace_size(None, None) == M.MOE_ERR_INVALID_ARG
    for missing in ("x", "W", "y", "off"):          # several groups need offsets
        assert _fwd(lib, s, **{missing: None}) == M.MOE_ERR_INVALID_ARG, missing
    for odd in ("x", "W", "y", "res", "z", "bias"):
        assert _fwd(lib, s, **{odd: FAKE + 8}) == M.MOE_ERR_INVALID_ARG, odd
    for missing in ("x", "W", "z", "dy", "off"):
        assert _bwd(lib, s, **{missing: None}) == M.MOE_ERR_INVALID_ARG, missing
    assert _bwd(lib, s, dx=None, dW=None, db=None) == M.MOE_ERR_INVALID_ARG
    for odd in ("x", "W", "z", "dy", "dx", "dW", "db"):
        assert _bwd(lib, s, **{odd: FAKE + 8}) == M.MOE_ERR_INVALID_ARG, odd
    n = M.moe_linear_workspace_size(s)
    assert _bwd(lib, s, n=n - 1) == M.MOE_ERR_WORKSPACE
    assert _bwd(lib, s, ws=None) == M.MOE_ERR_WORKSPACE
    assert _bwd(lib, s, ws=FAKE + 16) == M.MOE_ERR_WORKSPACE
    # no rows: a valid no-op (nothing to write either)
    e = M.make_linear(0, 128, 256, E=8)
    assert _fwd(lib, e, x=None, W=None, y=None) == M.MOE_OK
    assert _bwd(lib, e, x=None, W=None, z=None, dy=None, dx=FAKE, dW=None, db=None) == M.MOE_OK


@pytest.mark.parametrize("dims", [(64, 64, 1), (4096, 768, 128), (512, 2048, 256)])
def test_workspace_never_shrinks_with_rows(lib, dims):
    di, do, E = dims
    for act in (M.MOE_ACT_NONE, M.MOE_ACT_SILU):
        prev = 0
        for rows in (0, 1, 2, 7, 63, 64, 65, 127, 128, 129, 255, 256, 300, 1000, 4096, 16384, 1 << 20):
            n = M.moe_linear_workspace_size(M.make_linear(rows, di, do, E=E, act=act))
            assert n >= prev and n % 256 == 0
            prev = n


def test_combine_refusals(lib):
    s = M.make_shape(64, 128, 128, 8, 2)
    f = lambda y=FAKE, slot=FAKE, w=FAKE, res=None, out=FAKE, sh=s: lib.moe_combine_rows(
        ctypes.byref(sh), y, slot, w, res, out, None, None)
    for kw in (dict(y=None), dict(slot=None), dict(out=None), dict(y=FAKE + 8), dict(out=FAKE + 4),
               dict(res=FAKE + 2), dict(slot=FAKE + 2), dict(w=FAKE + 1),
               dict(sh=M.make_shape(64, 100, 128, 8, 2)), dict(sh=M.make_shape(64, 128, 128, 8, 9))):
        assert f(**kw) == M.MOE_ERR_INVALID_ARG, kw
    assert f(y=None, slot=None, out=None, sh=M.make_shape(0, 128, 128, 8, 2)) == M.MOE_OK
    b = lambda dout=FAKE, y=FAKE, slot=FAKE, w=FAKE, dy=FAKE, dw=FAKE, sh=s: \
        lib.moe_combine_rows_backward(ctypes.byref(sh), dout, y, slot, w, dy, dw, None, None)
    for kw in (dict(dout=None), dict(slot=None), dict(dy=None, dw=None), dict(y=None),
               dict(dout=FAKE + 8), dict(y=FAKE + 8), dict(dy=FAKE + 8), dict(dw=FAKE + 2)):
        assert b(**kw) == M.MOE_ERR_INVALID_ARG, kw
    assert b(dout=None, slot=None, sh=M.make_shape(0, 128, 128, 8, 2)) == M.MOE_OK


def _lists(ptrs, numel, types):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*types))


def _clip(lib, ptrs, numel, types, outs=None, max_norm=1.0, norm=FAKE, ws=FAKE, nb=M.MOE_GRAD_WS_BYTES):
    p, c, t = _lists(ptrs, numel, types)
    o = None if outs is None else (ctypes.c_void_p * len(outs))(*outs)
    return lib.moe_clip_grads(len(ptrs), p, o, c, t, max_norm, norm, None, ws, nb, None)


def test_clip_refusals(lib):
    A, C = 1 << 20, 1 << 21
    f32, b16 = M.MOE_TYPE_F32, M.MOE_TYPE_BF16
    bad = M.MOE_ERR_INVALID_ARG
    assert _clip(lib, [A], [16], [7]) == bad                         # unknown type
    assert _clip(lib, [A], [-1], [f32]) == bad
    assert _clip(lib, [A], [(1 << 40) + 1], [f32]) == bad
    assert _clip(lib, [None], [1], [f32]) == bad
    assert _clip(lib, [A + 2], [4], [f32]) == bad                    # not aligned to its elements
    assert _clip(lib, [A + 1], [4], [b16]) == bad
    assert _clip(lib, [A], [4], [f32], norm=None) == bad
    for m in (0.0, -1.0, float("nan")):
        assert _clip(lib, [A], [4], [f32], max_norm=m) == bad, m
    # overlaps: the same tensor twice, a view into another, an output on another's input
    assert _clip(lib, [A, A], [16, 16], [f32, f32]) == bad
    assert _clip(lib, [A, A + 32], [16, 16], [f32, f32]) == bad
    assert _clip(lib, [A, C], [16, 16], [f32, f32], outs=[C, A]) == bad
    assert _clip(lib, [A], [16], [f32], outs=[A + 4]) == bad
    many = [A + 64 * i for i in range(300)]
    assert _clip(lib, many + [many[7]], [16] * 301, [f32] * 301) == bad
    # neighbours and empty tensors do not overlap: the call gets as far as the workspace
    assert _clip(lib, [A, A + 64, None], [16, 16, 0], [f32, f32, f32], ws=None) == M.MOE_ERR_WORKSPACE
    assert _clip(lib, [A], [16], [f32], nb=M.MOE_GRAD_WS_BYTES - 1) == M.MOE_ERR_WORKSPACE
    assert _clip(lib, [A], [16], [f32], ws=FAKE + 8) == M.MOE_ERR_WORKSPACE
    p, c, t = _lists([A], [4], [f32])
    assert lib.moe_grad_norm(-1, p, c, t, FAKE, None, FAKE, 1 << 20, None) == bad
    assert lib.moe_grad_norm((1 << 20) + 1, p, c, t, FAKE, None, FAKE, 1 << 20, None) == bad
    assert lib.moe_grad_norm(1, None, c, t, FAKE, None, FAKE, 1 << 20, None) == bad
    assert lib.moe_grad_norm(1, p, c, t, FAKE, None, FAKE, 16, None) == M.MOE_ERR_WORKSPACE


def test_binding_checks_before_the_library():
    """Wrong places, shapes, types and devices raise in the binding."""
    cpu = torch.zeros(4, 8, dtype=torch.bfloat16)
    s = M.make_linear(4, 8, 8)
    with pytest.raises(ValueError, match="CUDA"):
        M.moe_linear_forward(s, cpu, None, torch.zeros(8, 8, dtype=torch.bfloat16), None, None, cpu)
    with pytest.raises(ValueError, match="W: expected shape"):
        M.moe_linear_forward(s, cpu, None, torch.zeros(4, 8, dtype=torch.bfloat16), None, None, cpu)
    with pytest.raises(ValueError, match="expert_offsets"):
        M.moe_linear_backward(M.make_linear(4, 8, 8, E=4), cpu, torch.zeros(4, dtype=torch.int32),
                              None, None, cpu, None, None, None, None, None)
    with pytest.raises(ValueError, match="slot_pos"):
        M.moe_combine_rows(M.make_shape(4, 128, 128, 8, 2), None, torch.zeros(4, 3, dtype=torch.int32),
                           None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        M.moe_grad_norm([cpu], None)
    with pytest.raises(ValueError, match="outs"):
        M.moe_clip_grads([], 1.0, None, outs=[cpu])


class _Fake:
    """Stands in for a CUDA tensor on a given device in the device check."""
    is_cuda = True

    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_tensors_on_two_devices_are_refused(monkeypatch):
    monkeypatch.setattr(M.torch, "Tensor", _Fake)
    with pytest.raises(ValueError, match="different devices"):
        M._on_one_device(x=_Fake(0), W=_Fake(1))
