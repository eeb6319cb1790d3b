"""Operators around the routed layer, measured: the linear product with bias,
activation and residual (dense, and grouped by expert with ragged sizes), the
combine of bf16 expert rows, and the global gradient norm with clipping; each
with its gradient where it has one.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes a case's inputs on the GPU from a seed, and ``run()`` is one
pass: the plain form in elementary fp32 torch operations, or, with ``own`` set,
the library's calls. ``exact()`` is the same result from the definition in fp64.
"""
import math

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # one token through a dense up projection: the weights are read once (d and d_ff of the decode workload)
        dict(name="linear_token", op="linear", rows=1, d_in=4096, d_out=14336, E=1, act="gelu",
             bias=True, residual=False, save_z=False, backward=False),
        # a handful of tokens through a small layer: launch latency
        dict(name="linear_small", op="linear", rows=100, d_in=256, d_out=384, E=1, act="relu",
             bias=True, residual=True, save_z=True, backward=False),
        # a long prompt through the down projection, added to the residual stream
        dict(name="linear_prompt", op="linear", rows=16384, d_in=14336, d_out=4096, E=1, act="none",
             bias=True, residual=True, save_z=False, backward=False),
        # a training step's backward through a dense layer
        dict(name="linear_train", op="linear", rows=4096, d_in=2048, d_out=4096, E=1, act="gelu_tanh",
             bias=True, residual=False, save_z=True, backward=True),
        # one token's two experts (decode workload)
        dict(name="experts_token", op="linear", rows=2, d_in=4096, d_out=14336, E=8, k=2, capacity=0,
             zipf=0.0, act="silu", bias=True, residual=False, save_z=False, backward=False),
        # fine-grained experts with a skewed load: from thousands of rows to a few (fine_grained workload)
        dict(name="experts_fine", op="linear", rows=65536, d_in=7168, d_out=2048, E=256, k=8, capacity=0,
             zipf=1.1, act="relu", bias=False, residual=False, save_z=False, backward=False),
        # experts with a capacity: rows behind the kept ones belong to no expert (capacity workload)
        dict(name="experts_capacity", op="linear", rows=32768, d_in=2048, d_out=768, E=128, k=8, capacity=320,
             zipf=1.0, act="gelu", bias=True, residual=False, save_z=True, backward=False),
        # the same layer's backward
        dict(name="experts_train", op="linear", rows=32768, d_in=2048, d_out=768, E=128, k=8, capacity=320,
             zipf=1.0, act="gelu", bias=True, residual=False, save_z=True, backward=True),
        # the weighted combine of a prompt's expert rows into the residual stream (prefill workload)
        dict(name="combine_prompt", op="combine", T=16384, d=4096, E=8, k=2, capacity=0, zipf=0.0,
             residual=True, backward=False),
        # its backward, with dropped assignments
        dict(name="combine_train", op="combine", T=4096, d=2048, E=128, k=8, capacity=320, zipf=1.0,
             residual=False, backward=True),
        # the gradients of a small layer, norm below the limit: nothing is scaled, latency counts
        dict(name="clip_small", op="clip", sizes="524288,262144,1024,8", dtypes="f32,f32,f32,f32",
             ratio=0.5, inplace=True),
        # a whole layer's expert gradients, norm above the limit, into the optimizer's buffers
        dict(name="clip_layer", op="clip", sizes="402653184,201326592,262144,128,201326591,2049",
             dtypes="f32,f32,f32,f32,bf16,bf16", ratio=3.0, inplace=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "grouped", "grouped", "grouped", "combine", "clip"])
    if op in ("linear", "grouped"):
        while True:
            c = dict(op="linear", d_in=8 * _log(rng, 8, 1792), d_out=8 * _log(rng, 8, 1792),
                     act=rng.choice(ACTS), bias=rng.random() < 0.7, backward=rng.random() < 0.4)
            if op == "linear":
                c |= dict(E=1, rows=_log(rng, 1, 16384))
            else:
                E = _log(rng, 2, 256)
                k = rng.randint(1, min(E, 8))
                T = _log(rng, 1, 8192)
                c |= dict(E=E, k=k, rows=T * k, zipf=rng.choice([0.0, 0.5, 1.0, 1.1]),
                          capacity=rng.choice([0, 0, max(1, math.ceil(1.25 * T * k / E))]))
            c["residual"] = not c["backward"] and rng.random() < 0.4
            c["save_z"] = c["act"] != "none" and (c["backward"] or rng.random() < 0.4)
            flops = (2 if c["backward"] else 1) * 2 * c["rows"] * c["d_in"] * c["d_out"]
            if flops <= 1.0e12 and c["E"] * c["d_in"] * c["d_out"] <= 1 << 31 and c["rows"] * max(c["d_in"], c["d_out"]) <= 1 << 28:
                return c
    if op == "combine":
        while True:
            E = _log(rng, 2, 256)
            k = rng.randint(1, min(E, 8))
            T = _log(rng, 1, 16384)
            d = 128 * _log(rng, 1, 56)
            if T * k * d <= 1 << 28:
                return dict(op="combine", T=T, d=d, E=E, k=k, zipf=rng.choice([0.0, 1.0]),
                            capacity=rng.choice([0, max(1, math.ceil(1.25 * T * k / E))]),
                            residual=rng.random() < 0.5, backward=rng.random() < 0.5)
    n = _log(rng, 1, 200)
    total = _log(rng, 1000, 400_000_000)
    parts = [rng.random() ** 3 + 1e-6 for _ in range(n)]
    sizes = [max(1, int(total * p / sum(parts))) for p in parts]
    return dict(op="clip", sizes=",".join(map(str, sizes)),
                dtypes=",".join(rng.choice(["f32", "bf16"]) for _ in sizes),
                ratio=(r := rng.choice([0.5, 3.0, 40.0])), inplace=r < 1.0)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=BF16):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    if out.dim() < 3:
        return out.copy_(torch.randn(shape, generator=g, device="cuda").mul_(std))
    for part in out:          # one expert at a time: no fp32 copy of all of them
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(std))
    return out


def _choices(g, T, E, k, zipf):
    """T tokens' k distinct experts, drawn from a Zipf law over a random order of the experts."""
    order = torch.randperm(E, generator=g, device="cuda").add(1).to(F32)
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    return torch.topk(-zipf * torch.log(order) - torch.log(-torch.log(u)), k, dim=1).indices


def _dispatch(g, T, E, k, zipf, capacity):
    """Offsets [E+1] and slot_pos [T, k]: assignments grouped by expert in token order, those past the capacity dropped."""
    e = _choices(g, T, E, k, zipf).reshape(-1)
    counts = torch.bincount(e, minlength=E)
    kept = counts.clamp(max=capacity) if capacity > 0 else counts
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = kept.cumsum(0)
    by_expert = torch.argsort(e, stable=True)
    rank = torch.empty_like(e)
    rank[by_expert] = torch.arange(T * k, device="cuda") - (counts.cumsum(0) - counts)[e[by_expert]]
    slot = torch.where(rank < kept[e], offsets[e] + rank, -1)
    return offsets.to(I32), slot.reshape(T, k).to(I32)


def _ints(text):
    return [int(v) for v in text.split(",")]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "linear":
        rows, di, do, E = case["rows"], case["d_in"], case["d_out"], case["E"]
        if "k" in case:
            s["offsets"], _ = _dispatch(g, rows // case["k"], E, case["k"], case["zipf"], case["capacity"])
            s["bounds"] = s["offsets"].tolist()
        else:
            s["offsets"], s["bounds"] = None, [0, rows]
        s["x"] = _normal(g, rows, di)
        s["W"] = _normal(g, E, do, di, std=0.02)
        s["bias"] = _normal(g, E, do, std=0.1, dtype=F32) if case["bias"] else None
        if case["backward"]:
            s["z"] = _normal(g, rows, do) if case["act"] != "none" else None
            s["dy"] = _normal(g, rows, do, std=1e-3)
            s["dx"] = torch.zeros(rows, di, dtype=BF16, device="cuda")
            s["dW"] = torch.zeros(E, do, di, dtype=BF16, device="cuda")
            s["db"] = torch.zeros(E, do, dtype=F32, device="cuda") if case["bias"] else None
        else:
            s["R"] = _normal(g, rows, do) if case["residual"] else None
            s["z"] = torch.zeros(rows, do, dtype=BF16, device="cuda") if case["save_z"] else None
            s["y"] = torch.zeros(rows, do, dtype=BF16, device="cuda")
    elif case["op"] == "combine":
        T, d, k = case["T"], case["d"], case["k"]
        s["offsets"], s["slot"] = _dispatch(g, T, case["E"], k, case["zipf"], case["capacity"])
        s["w"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), dim=1)
        s["y"] = _normal(g, T * k, d)
        if case["backward"]:
            s["dout"] = _normal(g, T, d, std=1e-3)
            s["dy"] = torch.zeros(T * k, d, dtype=BF16, device="cuda")
            s["dw"] = torch.zeros(T, k, dtype=F32, device="cuda")
        else:
            s["R"] = _normal(g, T, d) if case["residual"] else None
            s["out"] = torch.zeros(T, d, dtype=BF16, device="cuda")
    else:
        sizes = _ints(case["sizes"])
        types = [F32 if t == "f32" else BF16 for t in case["dtypes"].split(",")]
        std = 1e-3
        s["grads"] = []
        for n, t in zip(sizes, types):
            grad = torch.empty(n, dtype=t, device="cuda")
            for part in grad.split(1 << 26):
                part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(std))
            s["grads"].append(grad)
        # the norm comes out near std * sqrt(n): `ratio` is how far above the limit it lies
        s["max_norm"] = std * math.sqrt(sum(sizes)) / case["ratio"]
        s["outs"] = None if case["inplace"] else [torch.zeros_like(v) for v in s["grads"]]
        s["norm"] = torch.zeros(1, dtype=F32, device="cuda")
    if own:
        from sparse_mixture_experts_17_b200 import moe as M
        s["M"] = M
        s["status"] = torch.zeros(1, dtype=I32, device="cuda")
        if case["op"] == "linear":
            act = getattr(M, "MOE_ACT_" + case["act"].upper())
            s["shape"] = M.make_linear(case["rows"], case["d_in"], case["d_out"], E=case["E"], act=act)
            if case["backward"]:
                s["ws"] = M.alloc_linear_workspace(s["shape"])
        elif case["op"] == "combine":
            s["shape"] = M.make_shape(case["T"], case["d"], 128, case["E"], case["k"], capacity=case["capacity"])
        else:
            s["ws"] = M.alloc_grad_workspace(s["grads"])
    return s


# ---------------------------------------------------------------- one pass

def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _plain_linear(s):
    """Group by group (a dense layer is one group): the groups' sizes differ too much for one padded batch."""
    c, b = s["case"], s["bounds"]
    groups = [(e, slice(b[e], b[e + 1])) for e in range(c["E"]) if b[e + 1] > b[e]]
    if not c["backward"]:
        for e, r in groups:
            z = s["x"][r].float() @ s["W"][e].float().T
            if s["bias"] is not None:
                z = z + s["bias"][e]
            if s["z"] is not None:
                s["z"][r] = z.to(BF16)
            y = _act(z, c["act"])
            s["y"][r] = (y if s["R"] is None else y + s["R"][r].float()).to(BF16)
        return {"y": s["y"]} | ({"z": s["z"]} if s["z"] is not None else {})
    s["dW"].zero_()
    if s["db"] is not None:
        s["db"].zero_()
    for e, r in groups:
        dz = s["dy"][r].float()
        if s["z"] is not None:
            dz = dz * _act_grad(s["z"][r].float(), c["act"])
        s["dx"][r] = (dz @ s["W"][e].float()).to(BF16)
        s["dW"][e] = (dz.T @ s["x"][r].float()).to(BF16)
        if s["db"] is not None:
            s["db"][e] = dz.sum(0)
    return {"dx": s["dx"], "dW": s["dW"]} | ({"db": s["db"]} if s["db"] is not None else {})


def _plain_combine(s):
    c = s["case"]
    kept = (s["slot"] >= 0).unsqueeze(-1)
    rows = s["slot"].clamp(min=0).long()
    if not c["backward"]:
        out = (s["w"].unsqueeze(-1) * torch.where(kept, s["y"][rows].float(), 0.0)).sum(1)
        s["out"].copy_(out if s["R"] is None else out + s["R"].float())
        return {"out": s["out"]}
    dout = s["dout"].float().unsqueeze(1)
    s["dw"].copy_((dout * torch.where(kept, s["y"][rows].float(), 0.0)).sum(-1))
    keep = kept.squeeze(-1)
    s["dy"][s["slot"][keep].long()] = (s["w"].unsqueeze(-1) * dout)[keep].to(BF16)
    return {"dy": s["dy"], "dw": s["dw"]}


def _plain_clip(s):
    norm = torch.stack([g.float().square().sum(dtype=F64) for g in s["grads"]]).sum().sqrt().float()
    s["norm"].copy_(norm)
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    outs = s["grads"] if s["outs"] is None else s["outs"]
    for g, o in zip(s["grads"], outs):
        o.copy_(g.float() * coef)
    return {"norm": s["norm"], "outs": outs}


def run(s):
    c = s["case"]
    if not own:
        return {"linear": _plain_linear, "combine": _plain_combine, "clip": _plain_clip}[c["op"]](s)
    M = s["M"]
    if c["op"] == "linear":
        if c["backward"]:
            M.moe_linear_backward(s["shape"], s["x"], s["offsets"], s["W"], s["z"], s["dy"], s["dx"], s["dW"],
                                  s["db"], s["status"], s["ws"])
            return {"dx": s["dx"], "dW": s["dW"]} | ({"db": s["db"]} if s["db"] is not None else {})
        M.moe_linear_forward(s["shape"], s["x"], s["offsets"], s["W"], s["bias"], s["R"], s["y"], s["z"], s["status"])
        return {"y": s["y"]} | ({"z": s["z"]} if s["z"] is not None else {})
    if c["op"] == "combine":
        if c["backward"]:
            M.moe_combine_rows_backward(s["shape"], s["dout"], s["y"], s["slot"], s["w"], s["dy"], s["dw"], s["status"])
            return {"dy": s["dy"], "dw": s["dw"]}
        M.moe_combine_rows(s["shape"], s["y"], s["slot"], s["w"], s["R"], s["out"], s["status"])
        return {"out": s["out"]}
    M.moe_clip_grads(s["grads"], s["max_norm"], s["norm"], s["outs"], s["status"], s["ws"])
    return {"norm": s["norm"], "outs": s["grads"] if s["outs"] is None else s["outs"]}


# ---------------------------------------------------------------- what a pass cannot do without

def _expected_kept(case):
    """(rows in groups, groups with rows), in expectation over the draws of _choices."""
    if "k" not in case:
        return case.get("rows", 0), 1
    E, k = case["E"], case["k"]
    T = case["T"] if "T" in case else case["rows"] // k
    p = [r ** -case["zipf"] for r in range(1, E + 1)]
    # P(expert chosen) of k draws without replacement: 1 - exp(-c p) with c fitted so that they add up to k
    lo, hi = 0.0, 1e9
    for _ in range(100):
        mid = (lo + hi) / 2
        lo, hi = (mid, hi) if sum(1 - math.exp(-mid * v) for v in p) < k else (lo, mid)
    q = [1 - math.exp(-hi * v) for v in p]
    cap = case["capacity"] if case["capacity"] > 0 else T
    return sum(min(T * v, cap) for v in q), sum(1 - (1 - min(v, 1 - 1e-12)) ** T for v in q)


def work(case):
    if case["op"] == "linear":
        di, do, E = case["d_in"], case["d_out"], case["E"]
        n, used = _expected_kept(case)
        if case["backward"]:
            read = 2 * n * (di + do * (2 if case["act"] != "none" else 1)) + 2 * used * di * do
            return dict(bytes=read + 2 * n * di + 2 * E * di * do + (4 * E * do if case["bias"] else 0), flops=4 * n * di * do)
        read = 2 * n * di + 2 * used * di * do + (4 * used * do if case["bias"] else 0) + (2 * n * do if case["residual"] else 0)
        return dict(bytes=read + 2 * n * do * (2 if case["save_z"] else 1), flops=2 * n * di * do)
    if case["op"] == "combine":
        T, d, k = case["T"], case["d"], case["k"]
        n, _ = _expected_kept(case)
        if case["backward"]:
            return dict(bytes=2 * T * d + 4 * n * d + 12 * T * k, flops=3 * n * d)
        return dict(bytes=2 * T * d * (2 if case["residual"] else 1) + 2 * n * d + 8 * T * k, flops=2 * n * d)
    sizes = _ints(case["sizes"])
    total = sum(n * (4 if t == "f32" else 2) for n, t in zip(sizes, case["dtypes"].split(",")))
    return dict(bytes=total * (1 if case["inplace"] else 2), flops=3 * sum(sizes))


# ---------------------------------------------------------------- the definition in fp64

def _exact_act(z, act):
    """act(z) and act'(z): the derivative by autograd, the value from the definition."""
    z = z.detach().requires_grad_(True)
    with torch.enable_grad():
        if act == "none":
            y = z * 1.0
        elif act == "relu":
            y = torch.where(z > 0, z, torch.zeros_like(z))
        elif act == "gelu":
            y = z * torch.special.ndtr(z)
        elif act == "gelu_tanh":
            y = z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        else:
            y = z / (1 + torch.exp(-z))
        (d,) = torch.autograd.grad(y.sum(), z)
    return y.detach(), d


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        rows, di, do, E, b = case["rows"], case["d_in"], case["d_out"], case["E"], s["bounds"]
        step = max(1, (1 << 27) // max(di, do))      # rows at a time: bounded fp64 copies
        if case["backward"]:
            dx = torch.zeros(rows, di, dtype=F64, device="cuda")
            dW = torch.zeros(E, do, di, dtype=F64, device="cuda")
            db = torch.zeros(E, do, dtype=F64, device="cuda")
            for e in range(E):
                for a in range(b[e], b[e + 1], step):
                    r = slice(a, min(a + step, b[e + 1]))
                    dz = s["dy"][r].double()
                    if s["z"] is not None:
                        dz = dz * _exact_act(s["z"][r].double(), case["act"])[1]
                    dx[r] = torch.einsum("rn,nk->rk", dz, s["W"][e].double())
                    dW[e] += torch.einsum("rn,rk->nk", dz, s["x"][r].double())
                    db[e] += torch.einsum("rn->n", dz)
            return {"dx": dx, "dW": dW} | ({"db": db} if case["bias"] else {})
        y = torch.zeros(rows, do, dtype=F64, device="cuda")
        zs = torch.zeros(rows, do, dtype=F64, device="cuda") if case["save_z"] else None
        for e in range(E):
            for a in range(b[e], b[e + 1], step):
                r = slice(a, min(a + step, b[e + 1]))
                z = torch.einsum("rk,nk->rn", s["x"][r].double(), s["W"][e].double())
                if case["bias"]:
                    z += s["bias"][e].double()
                if zs is not None:
                    zs[r] = z
                y[r] = _exact_act(z, case["act"])[0]
                if case["residual"]:
                    y[r] += s["R"][r].double()
        return {"y": y} | ({"z": zs} if zs is not None else {})
    if case["op"] == "combine":
        T, d, k = case["T"], case["d"], case["k"]
        y64 = torch.cat([s["y"].double(), torch.zeros(1, d, dtype=F64, device="cuda")])   # slot -1: the zero row
        if case["backward"]:
            dy = torch.zeros(T * k + 1, d, dtype=F64, device="cuda")
            dw = torch.zeros(T, k, dtype=F64, device="cuda")
            for j in range(k):
                at = s["slot"][:, j].long()
                dw[:, j] = torch.einsum("td,td->t", s["dout"].double(), y64[at])
                dy[at] = s["w"][:, j:j + 1].double() * s["dout"].double()
            return {"dy": dy[:-1], "dw": dw}
        out = s["R"].double() if case["residual"] else torch.zeros(T, d, dtype=F64, device="cuda")
        for j in range(k):
            out += s["w"][:, j:j + 1].double() * y64[s["slot"][:, j].long()]
        return {"out": out}
    total = sum(float(torch.linalg.vector_norm(part.double()) ** 2) for g in s["grads"] for part in g.split(1 << 26))
    norm = math.sqrt(total)
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    return {"norm": torch.full((1,), norm, dtype=F64, device="cuda"), "outs": [g.double() * coef for g in s["grads"]]}
