"""Measured cases of the experts' products with 4-bit weights and of the head's loss.

Four operators: the two grouped products of the experts (gate/up with SwiGLU,
down) with weights held as 4-bit integers with one scale a group of columns,
and the softmax cross entropy of the output head over a large vocabulary
without its logits, forward and with its gradients.  Where ``own`` is false
they are computed in their plain form with elementary torch operations in 32
bits; where it is true, through the framework's entry points.
"""
import math

import torch

own = False

# the widths of the two layers: (D, F, Fs)
M1 = dict(D=4096, F=1024, Fs=1024)
XS2 = dict(D=2048, F=512, Fs=512)


def listed():
    return [
        # one sequence, one new token at the M.1 widths: nine experts' weights, latency
        dict(name="gate_up_token_m1", op="gate_up", T=1, E=256, k=8, **M1, group=128, popularity="uniform"),
        # a decode step of 32 sequences whose experts are unevenly popular
        dict(name="gate_up_decode_m1", op="gate_up", T=32, E=256, k=8, **M1, group=128, popularity="zipf"),
        # the same step's second product
        dict(name="down_decode_m1", op="down", T=32, E=256, k=8, **M1, group=128, popularity="zipf"),
        # an odd number of sequences on fine groups, no shared expert
        dict(name="down_odd_xs2", op="down", T=77, E=256, k=8, D=2048, F=512, Fs=0, group=32, popularity="uniform"),
        # a prefill chunk at the XS.2 widths: 128 rows an expert, ragged
        dict(name="gate_up_chunk_xs2", op="gate_up", T=4096, E=256, k=8, **XS2, group=64, popularity="uniform"),
        # a long prefill chunk at the M.1 widths, second product: 256 rows an expert
        dict(name="down_prefill_m1", op="down", T=8192, E=256, k=8, **M1, group=128, popularity="uniform"),
        # one token's score under M.1's head: the vocabulary's weights once
        dict(name="loss_fwd_token_m1", op="loss_fwd", rows=1, D=4096, vocab=100352, ignored=0.0),
        # a validation batch of short ragged sequences, odd vocabulary, padding ignored
        dict(name="loss_fwd_odd", op="loss_fwd", rows=999, D=2048, vocab=50021, ignored=0.1),
        # the M.1 training batch
        dict(name="loss_fwd_m1", op="loss_fwd", rows=8192, D=4096, vocab=100352, ignored=0.0625),
        # a small ragged batch with an odd vocabulary and a width past whole tiles
        dict(name="loss_bwd_odd", op="loss_bwd", rows=333, D=1000, vocab=33001, ignored=0.1),
        # the XS.2 training batch, padded
        dict(name="loss_bwd_xs2", op="loss_bwd", rows=4096, D=2048, vocab=100352, ignored=0.0625),
        # the M.1 training batch
        dict(name="loss_bwd_m1", op="loss_bwd", rows=8192, D=4096, vocab=100352, ignored=0.0625),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate_up", "down", "loss_fwd", "loss_bwd"])
    if op in ("gate_up", "down"):
        D, F = 256 * _log(rng, 1, 16), 256 * _log(rng, 1, 8)
        E = min(_log(rng, 8, 256), max(8, 256 * 4096 * 1024 // (D * F)))
        k = rng.randint(1, 8)
        T = _log(rng, 1, max(1, min(8192, 8192 * 8 * 4096 * 1024 // (k * D * F))))
        return dict(op=op, T=T, E=E, k=k, D=D, F=F, Fs=rng.choice([0, 256, F]), group=rng.choice([32, 64, 128]),
                    popularity=rng.choice(["uniform", "zipf"]))
    D = 8 * _log(rng, 8, 512)
    vocab = _log(rng, 500, 131072)
    rows = _log(rng, 1, max(1, min(16384, 8192 * 4096 * 100352 // (D * vocab))))
    return dict(op=op, rows=rows, D=D, vocab=vocab, ignored=rng.choice([0.0, 0.1, 0.5]))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ inputs

def _weights(g, count, rows, cols, group):
    """4-bit codes, two a byte (column 2j in the low half), and their scales, as a
    symmetric quantisation of normally distributed weights gives them."""
    codes = torch.empty(count, rows, cols // 2, dtype=torch.uint8, device="cuda")
    for c, part in zip(codes.split(32), range(0, count, 32)):
        v = torch.randn(min(32, count - part), rows, cols, generator=g, device="cuda")
        v = v.mul_(2.6).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        c.copy_(v[..., 0::2] | (v[..., 1::2] << 4))
    scales = 0.02 / 2.6 * (1.0 + 0.2 * torch.randn(count, rows, cols // group, generator=g, device="cuda"))
    return codes, scales.to(torch.bfloat16)


def _routing(g, T, E, k, popularity):
    """offsets [E + 1] and sorted_token [T k] of a batch: k distinct experts a token."""
    score = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp_(1e-30, 1 - 1e-7)))
    if popularity == "zipf":
        rank = torch.randperm(E, generator=g, device="cuda") + 1.0
        score = score - 1.2 * rank.log()
    chosen = score.topk(k, 1).indices.reshape(-1)
    order = torch.argsort(chosen, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(chosen, minlength=E).cumsum(0)
    return offsets, (order // k).to(torch.int32)


def _inputs(case, seed):
    g = _gen(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    st = dict(case)
    if case["op"] in ("gate_up", "down"):
        T, E, k, D, F, Fs, group = (case[n] for n in ("T", "E", "k", "D", "F", "Fs", "group"))
        st["offsets"], st["sorted_token"] = _routing(g, T, E, k, case["popularity"])
        # the most rows any expert has, as a program that pads its batch knows it
        st["most"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())
        if case["op"] == "gate_up":
            # normalised tokens, a few of them with outlier channels
            x = randn(T, D)
            x[:, : 8] *= 1.0 + 49.0 * (torch.rand(T, 1, generator=g, device="cuda") < 0.1)
            st["x"] = x.to(torch.bfloat16)
            st["w"], st["s"] = _weights(g, E, 2 * F, D, group)
            st["ws"], st["ss"] = _weights(g, 1, 2 * Fs, D, group) if Fs else (None, None)
        else:
            # what SwiGLU leaves: routed rows in expert order, then the shared expert's
            a, b = randn(T * k * F + T * Fs), randn(T * k * F + T * Fs)
            st["h"] = (a / (1.0 + torch.exp(-a)) * b).to(torch.bfloat16)
            st["w"], st["s"] = _weights(g, E, D, F, group)
            st["ws"], st["ss"] = _weights(g, 1, D, Fs, group) if Fs else (None, None)
        return st
    T, D, V = case["rows"], case["D"], case["vocab"]
    w = randn(V, D).mul_(0.02).to(torch.bfloat16)
    target = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    # hidden states that know their target to different degrees
    wt = w[target.long()].float()
    x = randn(T, D) + 14.0 * torch.rand(T, 1, generator=g, device="cuda") * wt / wt.square().sum(1, keepdim=True)
    if case["ignored"]:
        target[torch.rand(T, generator=g, device="cuda") < case["ignored"]] = -1
    st.update(x=x.to(torch.bfloat16), w=w, target=target)
    if case["op"] == "loss_bwd":
        # what the forward pass left, and the weight of each token in the mean
        st["lse"] = torch.cat([torch.logsumexp(p.float() @ w.float().T, 1) for p in st["x"].split(4096)])
        st["lse"][target < 0] = 0.0
        st["dloss"] = (0.5 + torch.rand(T, generator=g, device="cuda")) / T
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    if case["op"] in ("gate_up", "down"):
        T, E, k, D, F, Fs = (case[n] for n in ("T", "E", "k", "D", "F", "Fs"))
        if own:
            # the weights in the layout of the products, once, as a program does that loads them
            from mixture_experts_transformer_moe_amd import binding as b
            st["shape"] = b.moe_shape(T, D, E, k, F, Fs, 1.0, b.MOE_BF16)
            st["w"] = b.pack_int4(st["w"])
            st["ws"] = b.pack_int4(st["ws"]) if Fs else None
        if case["op"] == "gate_up":
            st["out"] = torch.empty(T * k * F + T * Fs, **bf)
        else:
            st["out"] = torch.empty(T * k, D, **bf)
            st["out_shared"] = torch.empty(T, D, **bf) if Fs else None
        return st
    if case["op"] == "loss_fwd":
        st["loss"], st["out_lse"] = torch.empty(case["rows"], **f32), torch.empty(case["rows"], **f32)
    else:
        st["dx"], st["dw"] = torch.empty_like(st["x"]), torch.empty_like(st["w"])
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


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    from mixture_experts_transformer_moe_amd import binding as b
    if s["op"] == "gate_up":
        b.moe_grouped_gate_up_int4(s["shape"], s["group"], None, s["sorted_token"], s["x"], s["offsets"], s["w"],
                                   s["s"], s["ws"], s["ss"], s["out"])
        n = s["T"] * s["k"] * s["F"]
        return {"h": s["out"][:n], "shared": s["out"][n:] if s["Fs"] else None}
    if s["op"] == "down":
        b.moe_grouped_down_int4(s["shape"], s["group"], s["h"], s["offsets"], s["w"], s["s"], s["ws"], s["ss"],
                                s["out"], s["out_shared"])
        return {"y": s["out"], "shared": s["out_shared"]}
    ws = _workspace(b.moe_head_loss_workspace_bytes(s["rows"], s["D"], s["vocab"]))
    if s["op"] == "loss_fwd":
        b.moe_head_loss_forward(s["x"], s["w"], s["target"], s["loss"], s["out_lse"], ws)
        return {"loss": s["loss"], "lse": s["out_lse"]}
    b.moe_head_loss_backward(s["x"], s["w"], s["target"], s["lse"], s["dloss"], s["dx"], s["dw"], ws)
    return {"dx": s["dx"], "dw": s["dw"]}


# ------------------------------------------------------------------ the plain forms

def _dequantise(codes, scales, group):
    """float32 weights [count, rows, cols] of codes and scales."""
    count, rows, half = codes.shape
    v = torch.stack([codes & 15, codes >> 4], 3).float() - 8.0
    v = v.reshape(count, rows, 2 * half // group, group) * scales.float()[..., None]
    return v.reshape(count, rows, 2 * half)


def _grouped(rows, offsets, most, codes, scales, group):
    """rows [S, K] in expert order, each by its expert's matrix [N, K], in float32."""
    at = torch.arange(rows.shape[0], device="cuda", dtype=torch.int32)
    e = torch.searchsorted(offsets[1:].contiguous(), at, right=True)
    if rows.shape[0] < codes.shape[0]:
        # fewer rows than experts: each row's own matrix
        return torch.bmm(_dequantise(codes[e], scales[e], group), rows.float()[:, :, None])[:, :, 0]
    place = (at - offsets[e]).long()
    padded = torch.zeros(codes.shape[0], most, rows.shape[1], device="cuda")
    padded[e, place] = rows.float()
    return torch.bmm(padded, _dequantise(codes, scales, group).mT)[e, place]


def _swiglu(y):
    gate, up = y.chunk(2, 1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _gate_up_plain(s):
    rows = s["x"][s["sorted_token"].long()]
    h = _swiglu(_grouped(rows, s["offsets"], s["most"], s["w"], s["s"], s["group"]))
    shared = None
    if s["Fs"]:
        shared = _swiglu(s["x"].float() @ _dequantise(s["ws"], s["ss"], s["group"])[0].T).to(torch.bfloat16).reshape(-1)
    return {"h": h.to(torch.bfloat16).reshape(-1), "shared": shared}


def _down_plain(s):
    n = s["T"] * s["k"] * s["F"]
    y = _grouped(s["h"][:n].view(-1, s["F"]), s["offsets"], s["most"], s["w"], s["s"], s["group"])
    shared = None
    if s["Fs"]:
        hs = s["h"][n:].view(s["T"], s["Fs"]).float()
        shared = (hs @ _dequantise(s["ws"], s["ss"], s["group"])[0].T).to(torch.bfloat16)
    return {"y": y.to(torch.bfloat16), "shared": shared}


def _loss_fwd_plain(s):
    z = s["x"].float() @ s["w"].float().T
    top = z.max(1, keepdim=True).values
    lse = torch.log(torch.exp(z - top).sum(1)) + top[:, 0]
    counts = s["target"] >= 0
    zt = z.gather(1, s["target"].clamp(min=0).long()[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return {"loss": torch.where(counts, lse - zt, zero), "lse": torch.where(counts, lse, zero)}


def _loss_bwd_plain(s):
    x, w = s["x"].float(), s["w"].float()
    p = torch.exp(x @ w.T - s["lse"][:, None])
    t = s["target"].clamp(min=0).long()
    p[torch.arange(p.shape[0], device="cuda"), t] -= 1.0
    p = p * torch.where(s["target"] >= 0, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    return {"dx": (p @ w).to(torch.bfloat16), "dw": (p.T @ x).to(torch.bfloat16)}


def run(state):
    if own:
        return _run_own(state)
    return {"gate_up": _gate_up_plain, "down": _down_plain, "loss_fwd": _loss_fwd_plain,
            "loss_bwd": _loss_bwd_plain}[state["op"]](state)


# ------------------------------------------------------------------ the least work

def _touched(case):
    """Experts that a batch uses, on average."""
    E, k, T = case["E"], case["k"], case["T"]
    p = [(i + 1) ** -1.2 if case["popularity"] == "zipf" else 1.0 for i in range(E)]
    total = sum(p)
    # the chance that an expert is among the k distinct ones of a token, scaled so that they sum to k
    lo, hi = 0.0, 1e9
    for _ in range(200):
        mid = 0.5 * (lo + hi)
        if sum(1.0 - math.exp(-mid * q / total) for q in p) < k:
            lo = mid
        else:
            hi = mid
    return sum(1.0 - math.exp(-lo * q / total * T) for q in p)


def work(case):
    if case["op"] in ("gate_up", "down"):
        T, k, D, F, Fs, G = (case[n] for n in ("T", "k", "D", "F", "Fs", "group"))
        up = case["op"] == "gate_up"
        a = 2 if up else 1                                     # matrices of F x D a call reads of each expert
        weights = a * D * (_touched(case) * F + Fs) * (0.5 + 2.0 / G)
        if up:
            rows = 2.0 * (T * D + T * k * F + T * Fs)
        else:
            rows = 2.0 * (T * k * F + T * Fs + T * k * D + (T * D if Fs else 0))
        return {"bytes": weights + rows, "flops": 2.0 * a * D * T * (k * F + Fs)}
    T, D, V = case["rows"], case["D"], case["vocab"]
    if case["op"] == "loss_fwd":
        return {"bytes": 2.0 * (T + V) * D + 12.0 * T, "flops": 2.0 * T * D * V}
    return {"bytes": 4.0 * (T + V) * D + 12.0 * T, "flops": 6.0 * T * D * V}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if s["op"] in ("gate_up", "down"):
        def matrix(codes, scales):
            v = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device="cuda")
            v[:, 0::2], v[:, 1::2] = (codes % 16).double(), (codes // 16).double()
            return (v - 8.0) * scales.double().repeat_interleave(s["group"], 1)

        def product(rows, m):
            y = rows.double() @ m.T
            if s["op"] == "down":
                return y
            half = y.shape[1] // 2
            return y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]

        if s["op"] == "gate_up":
            rows, shared = s["x"][s["sorted_token"].long()], s["x"]
        else:
            n = s["T"] * s["k"] * s["F"]
            rows, shared = s["h"][:n].reshape(-1, s["F"]), s["h"][n:].reshape(s["T"], -1)
        ends = s["offsets"].tolist()
        out = torch.cat([product(rows[ends[e]:ends[e + 1]], matrix(s["w"][e], s["s"][e])) for e in range(s["E"])
                         if ends[e + 1] > ends[e]])
        more = product(shared, matrix(s["ws"][0], s["ss"][0])) if s["Fs"] else None
        if s["op"] == "down":
            return {"y": out, "shared": more}
        return {"h": out.reshape(-1), "shared": None if more is None else more.reshape(-1)}
    w, counts = s["w"].double(), s["target"] >= 0
    if s["op"] == "loss_fwd":
        lse, loss = [], []
        for x, t in zip(s["x"].split(2048), s["target"].split(2048)):
            logp = torch.log_softmax(x.double() @ w.T, 1)
            first = (x.double() * w[0]).sum(1)
            lse.append(first - logp[:, 0])
            loss.append(-logp.gather(1, t.long().clamp(min=0)[:, None])[:, 0])
        lse, loss = torch.cat(lse), torch.cat(loss)
        return {"loss": loss.masked_fill(~counts, 0.0), "lse": lse.masked_fill(~counts, 0.0)}
    dx, dw = [], torch.zeros_like(w)
    for i in range(0, s["rows"], 2048):
        x, t = s["x"][i:i + 2048].double(), s["target"][i:i + 2048].long()
        scale = s["dloss"][i:i + 2048].double() * (t >= 0)
        d = torch.exp(x @ w.T - s["lse"][i:i + 2048].double()[:, None])
        d.scatter_add_(1, t.clamp(min=0)[:, None], torch.full_like(scale, -1.0)[:, None])
        d *= scale[:, None]
        dx.append(d @ w)
        dw.addmm_(d.T, x)
    return {"dx": torch.cat(dx), "dw": dw}
