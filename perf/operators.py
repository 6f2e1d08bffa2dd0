"""Measured cases of the training-side operators beside the MoE layer.

Three operators: the block's pre-norm (RMS norm or layer norm, with the residual
addition before it), its backward pass with the reduction of the weight's
gradient, and the orthogonalised update of a weight matrix (Newton-Schulz
products, with the momentum before them).  Where ``own`` is false they are
computed in their plain form with elementary torch operations in 32 bits;
where it is true, through the framework's entry points.
"""
import math

import torch

own = False

EPS_NORM = 1e-6
EPS_ORTH = 1e-7
MU = 0.95
A, B, C = 3.4445, -4.7750, 2.0315     # the quintic's coefficients


def listed():
    return [
        # 32 sequences, one new token each, at the M.1 width: latency
        dict(name="norm_fwd_decode", op="norm_fwd", kind="rms", rows=32, cols=4096, dtype="bf16", residual=True,
             affine="gamma"),
        # the long prefill chunk at the XS.2 width
        dict(name="norm_fwd_prefill", op="norm_fwd", kind="rms", rows=32768, cols=2048, dtype="bf16",
             residual=True, affine="gamma"),
        # fp32 activations with an odd width
        dict(name="norm_fwd_odd_f32", op="norm_fwd", kind="layer", rows=1000, cols=1023, dtype="f32",
             residual=False, affine="both"),
        # the XS.2 training batch, gradient of the residual stream joined
        dict(name="norm_bwd_xs2", op="norm_bwd", kind="rms", rows=4096, cols=2048, dtype="bf16", residual=True,
             affine="gamma"),
        # the M.1 batch with a full layer norm
        dict(name="norm_bwd_m1_layer", op="norm_bwd", kind="layer", rows=8192, cols=4096, dtype="bf16",
             residual=True, affine="both"),
        # a ragged fp32 batch with an odd width
        dict(name="norm_bwd_odd_f32", op="norm_bwd", kind="layer", rows=777, cols=1023, dtype="f32",
             residual=False, affine="both"),
        # the XS.2 router's weight (256 experts): one small fp32 matrix, latency
        dict(name="orth_router", op="orth", count=1, rows=256, cols=2048, dtype="f32", momentum=True,
             tokens=1024),
        # M.1's shared expert, down projection: one tall matrix
        dict(name="orth_shared_down_m1", op="orth", count=1, rows=4096, cols=1024, dtype="bf16", momentum=False,
             tokens=8192),
        # XS.2's down projections of one of eight expert-parallel ranks
        dict(name="orth_down_xs2_rank", op="orth", count=32, rows=2048, cols=512, dtype="bf16", momentum=True,
             tokens=1024),
        # odd sizes in fp32
        dict(name="orth_odd_f32", op="orth", count=7, rows=333, cols=1001, dtype="f32", momentum=False,
             tokens=500),
        # all of XS.2's gate/up projections: 128 tokens an expert
        dict(name="orth_gate_up_xs2", op="orth", count=256, rows=1024, cols=2048, dtype="bf16", momentum=False,
             tokens=128),
        # M.1's gate/up projections of one of eight expert-parallel ranks
        dict(name="orth_gate_up_m1_rank", op="orth", count=32, rows=2048, cols=4096, dtype="bf16",
             momentum=True, tokens=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "orth"])
    if op != "orth":
        cols = _log(rng, 64, 8192)
        rows = _log(rng, 1, min(32768, 8192 * 4096 // cols))
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        return dict(op=op, kind=rng.choice(["rms", "layer"]), rows=rows, cols=cols,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.5,
                    affine=rng.choice(["gamma", "both"]))
    rows, cols = _log(rng, 32, 4096), _log(rng, 32, 4096)
    if rng.random() < 0.5:
        rows, cols = (rows + 31) // 32 * 32, (cols + 31) // 32 * 32
    most = min(_orth_flops(256, 1024, 2048) / _orth_flops(1, rows, cols), 256 * 1024 * 2048 / (rows * cols), 256)
    count = _log(rng, 1, max(1, int(most)))
    return dict(op=op, count=count, rows=rows, cols=cols, dtype=rng.choice(["bf16", "f32"]),
                momentum=rng.random() < 0.5, tokens=_log(rng, 64, 4096))


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g = _gen(seed)
    dt = _dtype(case["dtype"])
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    st = dict(case)
    if case["op"] == "orth":
        n, r, c, k = case["count"], case["rows"], case["cols"], case["tokens"]
        # a weight gradient: the sum over the expert's tokens of outer products
        # of unequal weight, rounded as the weight-gradient kernels round it
        def grad():
            w = torch.logspace(0, -1.5, k, device="cuda")
            return (torch.bmm(randn(n, r, k) * w, randn(n, k, c)) * (1e-3 / math.sqrt(k))).to(dt)
        st["g"] = grad()
        st["out"] = torch.empty(n, r, c, dtype=torch.bfloat16, device="cuda")
        st["momentum"] = None
        if case["momentum"]:
            # what earlier steps left in the fp32 buffer, of full rank
            st["momentum"] = (randn(n, r, c) * torch.logspace(0, -1, c, device="cuda")).mul_(4e-3)
        return st
    T, D = case["rows"], case["cols"]
    # a residual stream: a few channels carry most of the energy
    chan = 1.0 + 20.0 * (torch.rand(D, generator=g, device="cuda") < 0.01)
    st["x"] = (randn(T, D) * chan + 0.25).to(dt)
    st["residual"] = (randn(T, D) * chan).to(dt) if case["residual"] else None
    st["gamma"] = 1.0 + 0.1 * randn(D)
    st["beta"] = 0.1 * randn(D) if case["affine"] == "both" else None
    f32 = dict(dtype=torch.float32, device="cuda")
    if case["op"] == "norm_fwd":
        st["y"] = torch.empty(T, D, dtype=dt, device="cuda")
        st["sum"] = torch.empty(T, D, dtype=dt, device="cuda") if case["residual"] else None
        st["mean"] = torch.empty(T, **f32) if case["kind"] == "layer" else None
        st["rstd"] = torch.empty(T, **f32)
        return st
    # backward: the forward's input and statistics, the upstream gradients
    xf = st["x"].double()
    st["mean"] = xf.mean(1).float() if case["kind"] == "layer" else None
    v = xf - xf.mean(1, keepdim=True) if case["kind"] == "layer" else xf
    st["rstd"] = (v.square().mean(1) + EPS_NORM).rsqrt().float()
    st["dy"] = randn(T, D).to(dt)
    st["dx"] = torch.empty(T, D, dtype=dt, device="cuda")
    st["dgamma"] = torch.empty(D, **f32)
    st["dbeta"] = torch.empty(D, **f32) if case["affine"] == "both" else None
    return st


# one workspace, kept by the program and shared by its calls (they follow each
# other on one stream)
_kept = {}


def _workspace(nbytes):
    if _kept.get("n", -1) < nbytes:
        _kept["ws"] = None
        _kept["ws"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
        _kept["n"] = nbytes
    return _kept["ws"]


def _run_own(s):
    from mixture_experts_transformer_moe_amd import binding as b
    if s["op"] == "orth":
        ws = _workspace(b.moe_orthogonalize_workspace_bytes(s["count"], s["rows"], s["cols"]))
        b.moe_orthogonalize(s["g"], s["momentum"], MU, True, 5, EPS_ORTH, 1.0, s["out"], ws)
        return {"out": s["out"], "momentum": s["momentum"]}
    kind = b.MOE_NORM_LAYER if s["kind"] == "layer" else b.MOE_NORM_RMS
    if s["op"] == "norm_fwd":
        b.moe_norm_forward(kind, s["x"], s["residual"], s["gamma"], s["beta"], EPS_NORM, s["sum"], s["y"],
                           s["mean"], s["rstd"])
        return {"y": s["y"], "sum": s["sum"], "mean": s["mean"], "rstd": s["rstd"]}
    ws = _workspace(b.moe_norm_workspace_bytes(s["rows"], s["cols"]))
    b.moe_norm_backward(kind, s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["residual"], s["dx"],
                        s["dgamma"], s["dbeta"], ws)
    return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}


def _ns_step(x):
    a = torch.bmm(x, x.mT)
    return A * x + torch.bmm(B * a + C * torch.bmm(a, a), x)


def _orth_plain(s):
    u = s["g"].float()
    if s["momentum"] is not None:
        s["momentum"].mul_(MU).add_(u)
        u = u + MU * s["momentum"]
    x = u.mT.contiguous() if s["rows"] > s["cols"] else u
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS_ORTH)
    x = _ns_step(_ns_step(_ns_step(_ns_step(_ns_step(x)))))
    x = x.mT.contiguous() if s["rows"] > s["cols"] else x
    return {"out": x.to(torch.bfloat16), "momentum": s["momentum"]}


def _norm_fwd_plain(s):
    dt = s["x"].dtype
    x = s["x"].float()
    total = None
    if s["residual"] is not None:
        total = (x + s["residual"].float()).to(dt)
        x = total.float()
    mean = x.mean(1) if s["kind"] == "layer" else None
    if mean is not None:
        x = x - mean[:, None]
    rstd = 1.0 / (x.square().mean(1) + EPS_NORM).sqrt()
    y = x * rstd[:, None] * s["gamma"]
    if s["beta"] is not None:
        y = y + s["beta"]
    return {"y": y.to(dt), "sum": total, "mean": mean, "rstd": rstd}


def _norm_bwd_plain(s):
    dt = s["x"].dtype
    x, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    h = (x - s["mean"][:, None]) * r if s["mean"] is not None else x * r
    g = dy * s["gamma"]
    dx = g - h * (g * h).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * r
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return {"dx": dx.to(dt), "dgamma": (dy * h).sum(0), "dbeta": dy.sum(0) if s["dbeta"] is not None else None}


def run(state):
    if own:
        return _run_own(state)
    return {"orth": _orth_plain, "norm_fwd": _norm_fwd_plain, "norm_bwd": _norm_bwd_plain}[state["op"]](state)


def _orth_flops(count, rows, cols):
    # five steps x <- (a I + b R + c R^2) x, R = x x^T, of an m x n matrix
    # (m <= n), taken as three and two: the second and third steps' R follow
    # from the first's by products of commuting symmetric m x m matrices (half
    # of each is computed), so that x enters 2 + 2 products: 6 m^2 n + 14 m^3
    m, n = min(rows, cols), max(rows, cols)
    return count * (6.0 * m * m * n + 14.0 * m ** 3)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "orth":
        n = case["count"] * case["rows"] * case["cols"]
        return {"bytes": n * (e + 2 + (8 if case["momentum"] else 0)),
                "flops": _orth_flops(case["count"], case["rows"], case["cols"])}
    n, T, D = case["rows"] * case["cols"], case["rows"], case["cols"]
    both, stats = case["affine"] == "both", 2 if case["kind"] == "layer" else 1
    if case["op"] == "norm_fwd":
        return {"bytes": n * e * (4 if case["residual"] else 2) + 4 * D * (1 + both) + 4 * T * stats, "flops": 8.0 * n}
    return {"bytes": n * e * (4 if case["residual"] else 3) + 4 * D * (2 + both) + 4 * T * stats, "flops": 14.0 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "orth":
        out, mom = [], []
        for i in range(s["count"]):      # one matrix at a time, Gram matrix on the short side
            u = s["g"][i].double()
            if s["momentum"] is not None:
                m = s["momentum"][i].double() * MU + u
                mom.append(m)
                u = u + MU * m
            x = u / (torch.linalg.matrix_norm(u) + EPS_ORTH)
            tall = x.shape[0] > x.shape[1]
            eye = torch.eye(min(x.shape), dtype=torch.float64, device="cuda")
            for _ in range(5):
                r = x.T @ x if tall else x @ x.T
                p = A * eye + r @ (B * eye + C * r)
                x = x @ p if tall else p @ x
            out.append(x)
        return {"out": torch.stack(out), "momentum": torch.stack(mom) if mom else None}
    x, gamma = s["x"].double(), s["gamma"].double()
    layer = s["kind"] == "layer"
    if s["op"] == "norm_fwd":
        total = None
        if s["residual"] is not None:
            total = x + s["residual"].double()
            # the norm reads the sum as it is stored
            x = (s["x"].float() + s["residual"].float()).to(s["x"].dtype).double()
        var, mean = torch.var_mean(x, 1, correction=0) if layer else (x.square().mean(1), None)
        rstd = (var + EPS_NORM) ** -0.5
        y = ((x - mean[:, None]) if layer else x) * (rstd[:, None] * gamma)
        if s["beta"] is not None:
            y = y + s["beta"].double()
        return {"y": y, "sum": total, "mean": mean, "rstd": rstd}
    dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
    h = ((x - s["mean"].double()[:, None]) if layer else x) * rstd
    t = dy * gamma
    along = (t * h).sum(1, keepdim=True) / x.shape[1]
    dx = t - h * along - (t.mean(1, keepdim=True) if layer else 0.0)
    dx = dx * rstd + (s["residual"].double() if s["residual"] is not None else 0.0)
    return {"dx": dx, "dgamma": torch.einsum("td,td->d", dy, h),
            "dbeta": dy.sum(0) if s["dbeta"] is not None else None}
