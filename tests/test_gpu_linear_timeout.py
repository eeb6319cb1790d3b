"""The bounded waits of the linear products, run out on the GPU without a fault or a hang.

With MOE_FLAG_TEST_TIMEOUT every wait is bounded at 50 ms, and the producer of one CTA of each cluster (the
only one, where a cluster is a single CTA) stops before the last block of its contraction. The block's
stage never fills: the MMA issue gives up on it after the MMAs of the blocks before have long been done,
the other producer finds no free stage, the epilogue no finished accumulator, and for dW the warp that
clears the last block's rows no block. Each sees the abort flag or its own limit and leaves; no copy and no
MMA is in flight by then. The call returns, the status holds MOE_ERR_TIMEOUT alone, and the next call in
the same process is right."""
import time

import pytest
import torch

from sparse_mixture_experts_17_b200 import moe as M
from test_gpu_linear import Case, sizes_to_offsets

pytestmark = pytest.mark.gpu
TIMEOUT = 1 << M.MOE_ERR_TIMEOUT


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_17_b200 import build
    build.build()


# rows, d_in, d_out, offsets: the engines and forms that the sizes choose, forward
FORWARD = {
    "split over a cluster": (1, 4096, 1024, None),
    "split, wider tile": (100, 2048, 1024, None),
    "unsplit": (100, 256, 384, None),
    "unsplit, groups": (60, 256, 384, sizes_to_offsets([7, 0, 33, 20])),
    "pairs": (2048, 512, 4096, None),
    "pairs, ragged groups": (2600, 520, 2056, sizes_to_offsets([900, 5, 0, 70, 1300, 300])),
    "pairs, double tiles": (4096, 2048, 4096, None),
}
# what is left out of the backward picks the kernels: dx, dW, both after dz and the bias sums
BACKWARD = {
    "dx on pairs": (2048, 4096, 512, None, dict(dW=False, db=False)),
    "dx split": (2, 1024, 4096, None, dict(dW=False, db=False)),
    "dW, whole last block": (640, 1024, 2048, None, dict(dx=False, db=False)),
    "dW, part of a last block": (611, 1024, 2048, None, dict(dx=False, db=False)),
    "dW in parts": (2100, 512, 512, None, dict(dx=False, db=False)),
    "all, ragged groups": (1600, 520, 1032, sizes_to_offsets([900, 0, 33, 600, 67]), {}),
}


def starved(c):
    s = c.shape
    return M.make_linear(s.rows, s.d_in, s.d_out, E=s.E, act=s.act, flags=M.MOE_FLAG_TEST_TIMEOUT)


def run_out(c, call):
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    st = int(c.status.item())
    assert st == TIMEOUT, st                # nothing else on the way
    assert 0.05 <= elapsed < 1.5, elapsed   # 50 ms waits, not the 2 s of production
    c.status.zero_()


@pytest.mark.parametrize("name", FORWARD)
def test_forward(name):
    rows, di, do, off = FORWARD[name]
    c = Case(rows, di, do, "silu", offsets=off, seed=rows)
    y, z = torch.empty_like(c.R), torch.empty_like(c.R)
    run_out(c, lambda: M.moe_linear_forward(starved(c), c.x, c.offsets, c.W, c.bias, c.R, y, z, c.status))
    c.check_forward(*c.forward())


@pytest.mark.parametrize("name", BACKWARD)
def test_backward(name):
    rows, di, do, off, left_out = BACKWARD[name]
    c = Case(rows, di, do, "gelu", offsets=off, seed=rows)
    ws = M.alloc_linear_workspace(c.shape)
    out = dict(dx=torch.empty_like(c.x), dW=torch.empty_like(c.W), db=torch.empty_like(c.bias))
    out = {k: None if k in left_out else v for k, v in out.items()}
    run_out(c, lambda: M.moe_linear_backward(starved(c), c.x, c.offsets, c.W, c.z, c.dy, out["dx"], out["dW"],
                                             out["db"], c.status, ws))
    c.check_backward(c.backward(ws=ws, **left_out))


def test_a_run_out_call_among_others():
    """On one stream, no wait between: a call that runs out leaves the calls before and behind it right."""
    c = Case(2048, 512, 1024, "gelu_tanh", seed=3)
    ref_y, ref = c.forward()[0], c.backward()
    ws = M.alloc_linear_workspace(c.shape)
    y = [torch.full_like(ref_y, 7.0) for _ in range(2)]
    o = [dict(dx=torch.empty_like(c.x), dW=torch.empty_like(c.W), db=torch.empty_like(c.bias)) for _ in range(2)]
    junk = dict(y=torch.empty_like(ref_y), dx=torch.empty_like(c.x), dW=torch.empty_like(c.W), db=torch.empty_like(c.bias))

    def calls():
        for i in range(2):
            M.moe_linear_forward(c.shape, c.x, None, c.W, c.bias, c.R, y[i], None, c.status)
            M.moe_linear_backward(c.shape, c.x, None, c.W, c.z, c.dy, o[i]["dx"], o[i]["dW"], o[i]["db"], c.status, ws)
            if i == 0:
                M.moe_linear_forward(starved(c), c.x, None, c.W, c.bias, c.R, junk["y"], None, c.status)
                M.moe_linear_backward(starved(c), c.x, None, c.W, c.z, c.dy, junk["dx"], junk["dW"], junk["db"],
                                      c.status, ws)
    run_out(c, calls)
    for i in range(2):
        assert torch.equal(y[i], ref_y)
        for k in ref:
            assert torch.equal(o[i][k], ref[k]), (i, k)
