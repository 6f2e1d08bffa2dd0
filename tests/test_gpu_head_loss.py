"""GPU parity of the head's loss and its gradients against the fp64 oracle
(oracle/loss_oracle.py), through the C ABI.

Tolerances.  u = 2^-24 is half a step of fp32, b = 2^-8 of bf16.
  * a logit: D exact products, added 16 at a time into the accumulator: D / 16 + 6
    roundings of sums that A = sum |x w| bounds: e = (D / 16 + 6) u A;
  * lse: the logits' e; the exponentials' own error, 2^-21 and 2 u of their
    argument, weighted by the probabilities (arguments past 40 weigh nothing): 5e-6;
    the sum's order, 64 values a lane, then 2 + 2 joins and a wave over the tiles: 100 u;
    the last roundings, 4 u |lse|.  loss: a second e and 4 u (|lse| + |z|);
  * P: p (e + 5e-6) and the two roundings before it is bf16, then b |P|;
  * dx = P w: P's errors e_P = (p (e + 5e-6) + 4 u) |g| add up with their signs
    known to none: at most sum e_P |w|.  The roundings to bf16 are independent, at
    most b |P| each: 8 standard deviations of b sqrt(sum P^2 w^2) / sqrt 3, taken as
    8 b / 1.7 of it.  The sum's order: (K / 16 + 6 + parts) u sum |P w|, and the
    output's own rounding b |dx|.  dw alike over the rows.
"""
import numpy as np
import pytest
import torch

from mixture_experts_transformer_moe_amd import binding as M
from oracle import loss_oracle as O
from oracle import update_oracle as U
from tests.gpu_common import say, to_f64

pytestmark = pytest.mark.gpu

u32, b16 = 2.0 ** -24, 2.0 ** -8


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).cuda()


def f32(a):
    return torch.from_numpy(np.asarray(a, np.float32)).cuda()


class Case:
    def __init__(self, rows, cols, vocab, ignored=0.2, seed=0, scale=1.0):
        rng = np.random.default_rng(seed)
        self.rows, self.cols, self.vocab = rows, cols, vocab
        w = rng.normal(size=(vocab, cols)) / np.sqrt(cols)
        y = rng.integers(0, vocab, rows)
        x = rng.normal(size=(rows, cols)) * 2 * scale + w[y] * 6 * rng.random((rows, 1)) * scale
        y[rng.random(rows) < ignored] = rng.choice([-1, -100, vocab, 2 ** 31 - 1])
        self.x, self.w, self.y = bf16(x), bf16(w), torch.from_numpy(y.astype(np.int32)).cuda()
        self.g = f32(rng.normal(size=rows) / max(rows, 1))
        # outputs inside guard bands
        self.guards = [torch.full((n + 256,), 7.0, dtype=dt, device="cuda")
                       for n, dt in ((rows, torch.float32), (rows, torch.float32), (rows * cols, torch.bfloat16),
                                     (vocab * cols, torch.bfloat16))]
        self.loss, self.lse = (self.guards[i][128:128 + rows] for i in (0, 1))
        self.dx = self.guards[2][128:128 + rows * cols].view(rows, cols)
        self.dw = self.guards[3][128:128 + vocab * cols].view(vocab, cols)
        n = M.moe_head_loss_workspace_bytes(rows, cols, vocab)
        self.ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")    # (NaN as any type)
        self.work = self.ws[256:256 + n]

    def forward(self, stream=None):
        M.moe_head_loss_forward(self.x, self.w, self.y, self.loss, self.lse, self.work, stream)

    def backward(self, dx=True, dw=True, stream=None):
        M.moe_head_loss_backward(self.x, self.w, self.y, self.lse, self.g, self.dx if dx else None,
                                 self.dw if dw else None, self.work, stream)

    def check_bands(self):
        for t in self.guards:
            assert (t[:128] == 7.0).all() and (t[-128:] == 7.0).all()
        assert (self.ws[:256] == 255).all() and (self.ws[-256:] == 255).all()

    def check_forward(self):
        x, w, y = to_f64(self.x), to_f64(self.w), self.y.cpu().numpy()
        loss, lse = O.forward(x, w, y)
        on = O.takes_part(y, self.vocab)
        got_loss, got_lse = to_f64(self.loss), to_f64(self.lse)
        assert (got_loss[~on] == 0).all() and (got_lse[~on] == 0).all()
        if not on.any():
            return
        self.e = np.zeros(self.rows)
        self.e[on] = (self.cols / 16 + 6) * u32 * (np.abs(x[on]) @ np.abs(w).T).max(1)
        z = lse - loss
        tol = self.e + 5e-6 + 100 * u32 + 4 * u32 * np.abs(lse)
        assert (np.abs(got_lse - lse)[on] <= tol[on]).all(), (np.abs(got_lse - lse)[on] / tol[on]).max()
        tol = tol + self.e + 4 * u32 * (np.abs(lse) + np.abs(z))
        assert (np.abs(got_loss - loss)[on] <= tol[on]).all(), (np.abs(got_loss - loss)[on] / tol[on]).max()

    def check_backward(self, dx=True, dw=True):
        x, w, y, lse, g = to_f64(self.x), to_f64(self.w), self.y.cpu().numpy(), to_f64(self.lse), to_f64(self.g)
        on = O.takes_part(y, self.vocab)
        x = np.where(on[:, None], x, 0.0)
        g, lse = np.where(on, g, 0.0), np.where(on, lse, 0.0)
        p = O.probs(x, w, y, lse, g)
        e = (self.cols / 16 + 6) * u32 * (np.abs(x) @ np.abs(w).T).max(1) + 5e-6
        q = np.abs(p) + (np.arange(self.vocab) == y[:, None]) * np.abs(g)[:, None]      # p g without the one
        ep = q * e[:, None] + 4 * u32 * np.abs(g)[:, None] * (q > 0)
        for want, got, a, ea, m, k in ((p @ w, self.dx, p, ep, w, self.vocab), (p.T @ x, self.dw, p.T, ep.T, x, self.rows)):
            if got is self.dx and not dx or got is self.dw and not dw:
                assert (got == 7.0).all()
                continue
            ma = np.abs(m)
            tol = ea @ ma + 8 * b16 / 1.7 * np.sqrt((a * a) @ (m * m)) + b16 * np.abs(want)
            tol += (k / 16 + 6 + 32) * u32 * (np.abs(a) @ ma) + 1e-37
            off = np.abs(to_f64(got) - want)
            assert (off <= tol).all(), f"{'dx' if got is self.dx else 'dw'}: worst {(off / tol).max():.2f}"
            if want.size > 1000 and np.linalg.norm(want) > 0:
                # the two roundings to bf16, each 2^-8 / sqrt 3 of a value at most on average
                assert np.linalg.norm(off) <= 1.5 * b16 * np.sqrt((want ** 2).sum() + ((a * a) @ (m * m)).sum())
        assert (to_f64(self.dx)[~on] == 0).all() or not dx


# every row tile (32, 64, 128, 256) inside and past its end, widths inside a stage, past
# one and over several, vocabularies of one column, inside a tile and past it
SIZES = [(1, 8, 1), (1, 64, 7), (2, 72, 257), (31, 200, 255), (32, 64, 256), (33, 128, 300), (64, 1000, 1000),
         (65, 256, 513), (100, 136, 2047), (128, 64, 64), (129, 192, 4099), (257, 8, 1000), (300, 520, 777),
         (513, 64, 3001), (700, 256, 2050)]


@pytest.mark.parametrize("rows,cols,vocab", SIZES)
def test_loss_and_gradients(rows, cols, vocab):
    say(f"head loss {rows} x {cols} over {vocab}")
    c = Case(rows, cols, vocab, seed=rows + cols)
    c.forward()
    torch.cuda.synchronize()
    c.check_forward()
    c.backward()
    torch.cuda.synchronize()
    c.check_backward()
    c.check_bands()


@pytest.mark.parametrize("rows", [20, 300])
def test_pieces_of_the_vocabulary(rows):
    # a width at which a piece holds 2048 columns: three pieces, the last ragged
    say(f"head loss in pieces, {rows} rows")
    c = Case(rows, 65536, 5003, seed=rows)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    c.check_forward()
    c.check_backward()
    c.check_bands()


def test_pieces_of_a_long_batch():
    # rows enough that a piece is shorter than the vocabulary (2^27 / 65536 columns);
    # against float64 on the GPU, a slice of rows and columns
    rows, cols, vocab = 65530, 64, 4500
    say(f"head loss {rows} x {cols} over {vocab}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(vocab, cols, generator=g, device="cuda").mul_(0.2).to(torch.bfloat16)
    y = torch.randint(-5, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(M.moe_head_loss_workspace_bytes(rows, cols, vocab), dtype=torch.uint8, device="cuda")
    dl = torch.full((rows,), 1.0 / rows, device="cuda")
    M.moe_head_loss_forward(x, w, y, loss, lse, ws)
    M.moe_head_loss_backward(x, w, y, lse, dl, dx, dw, ws)
    want = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 8192):
        xs, ys = x[i:i + 8192].double(), y[i:i + 8192].long()
        on = (ys >= 0).double()
        z = xs @ w.double().T
        s = torch.logsumexp(z, 1)
        assert ((lse[i:i + 8192] - s * on).abs() < 1e-5 * s.abs() + 2e-5).all()
        p = torch.exp(z - lse[i:i + 8192].double()[:, None])
        p.scatter_add_(1, ys.clamp(min=0)[:, None], -torch.ones_like(s)[:, None])
        p *= (on / rows)[:, None]
        want += p.T @ xs
        d = p @ w.double()
        assert (dx[i:i + 8192].double() - d).norm() <= 1.5 * b16 * d.norm()
    assert (dw.double() - want).norm() <= 1.5 * b16 * want.norm()


def test_only_one_gradient():
    c = Case(90, 128, 700, seed=3)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    both = c.dx.clone(), c.dw.clone()
    for dx, dw in ((True, False), (False, True)):
        for t in c.guards[2:]:
            t.fill_(7.0)
        c.backward(dx, dw)
        torch.cuda.synchronize()
        c.check_backward(dx, dw)
        assert torch.equal(c.dx if dx else c.dw, both[0] if dx else both[1])


@pytest.mark.parametrize("rows", [40, 300])
def test_rows_without_part_hold_anything(rows):
    c = Case(rows, 192, 600, ignored=0.4, seed=4)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    clean = [t.clone() for t in c.guards]
    off = (c.y < 0) | (c.y >= 600)
    assert off.any()
    n = int(off.sum())
    c.x[off] = torch.tensor([float("nan"), float("inf")], dtype=torch.bfloat16, device="cuda").repeat(n)[:n, None]
    c.forward()
    c.lse[off], c.g[off] = float("nan"), float("inf")
    c.backward()
    torch.cuda.synchronize()
    c.lse[off] = 0.0
    assert all(torch.equal(a, b) for a, b in zip(clean, c.guards))
    # no row at all
    c.y.fill_(-1)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    assert all((t == 0).all() for t in (c.loss, c.lse, c.dx, c.dw))


def test_bad_rows_stay_alone():
    c = Case(70, 64, 500, ignored=0.0, seed=5)
    c.forward()
    torch.cuda.synchronize()
    loss = c.loss.clone()
    c.x[3], c.x[5] = float("nan"), float("inf")
    c.forward()
    torch.cuda.synchronize()
    keep = torch.ones(70, dtype=torch.bool, device="cuda")
    keep[[3, 5]] = False
    assert torch.equal(c.loss[keep], loss[keep]) and not torch.isfinite(c.loss[~keep]).any()


@pytest.mark.parametrize("scale", [1e-3, 50.0])
def test_flat_and_peaked_rows(scale):
    # nearly uniform probabilities, and logits in the hundreds of which one is everything
    c = Case(150, 256, 900, seed=6, scale=scale)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    c.check_forward()
    c.check_backward()


def test_empty_batch():
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), bf16(np.ones((9, 64)))
    y, e = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    dw = torch.full((9, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    M.moe_head_loss_forward(x, w, y, e, e.clone(), None)
    M.moe_head_loss_backward(x, w, y, e, e, None, dw, None)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_repeats_bit_for_bit_on_streams_and_in_a_graph():
    cases = [Case(300, 128, 3000, seed=7), Case(50, 256, 1000, seed=8)]
    for c in cases:
        c.forward()
        c.backward()
    torch.cuda.synchronize()
    want = [[t.clone() for t in c.guards] for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for c, st in zip(cases, streams):
            for t in (c.loss, c.lse, c.dx, c.dw):
                t.zero_()
            st.wait_stream(torch.cuda.current_stream())
            c.forward(st)
            with torch.cuda.stream(st):
                c.backward()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, c in zip(want, cases) for a, b in zip(w, c.guards))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in cases:
            c.forward()
            c.backward()
    for i in range(3):
        for c in cases:
            for t in (c.loss, c.lse, c.dx, c.dw):
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, c in zip(want, cases) for a, b in zip(w, c.guards)), i
        cases[i % 2].forward()                           # eager work between the replays
        torch.cuda.synchronize()


def test_gradient_against_differences():
    # through the forward pass itself, on directions long enough to stand out of its rounding
    c = Case(40, 64, 300, ignored=0.1, seed=9)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    rng = np.random.default_rng(9)
    x, w, y, g = to_f64(c.x), to_f64(c.w), c.y.cpu().numpy(), to_f64(c.g)
    f = lambda x, w: (O.forward(x, w, y)[0] * g).sum()  # noqa: E731
    for a, d, of in ((x, to_f64(c.dx), 0), (w, to_f64(c.dw), 1)):
        v = rng.normal(size=a.shape)
        h = 1e-5
        diff = (f(x + h * v, w) - f(x - h * v, w) if of == 0 else f(x, w + h * v) - f(x, w - h * v)) / (2 * h)
        # independent roundings, two of b / sqrt 3 at most, over the direction: 6 deviations
        assert abs(diff - (d * v).sum()) <= 6 * 1.5 * b16 * np.linalg.norm(d * v) + 1e-6 * abs(diff)


def test_step_from_norm_to_update():
    # as a training step runs them: norm, loss, its gradients, the norm's backward, the head's update
    rows, cols, vocab = 200, 256, 512
    rng = np.random.default_rng(10)
    h, gamma = bf16(rng.normal(size=(rows, cols))), f32(1 + 0.1 * rng.normal(size=cols))
    w = bf16(rng.normal(size=(vocab, cols)) / 16)
    y = torch.from_numpy(rng.integers(-20, vocab, rows).astype(np.int32)).cuda()
    n = int((y >= 0).sum())
    x, rstd, dh = torch.empty_like(h), torch.empty(rows, device="cuda"), torch.empty_like(h)
    M.moe_norm_forward(M.MOE_NORM_RMS, h, None, gamma, None, 1e-6, None, x, None, rstd)
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ws = torch.empty(M.moe_head_loss_workspace_bytes(rows, cols, vocab), dtype=torch.uint8, device="cuda")
    M.moe_head_loss_forward(x, w, y, loss, lse, ws)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    M.moe_head_loss_backward(x, w, y, lse, torch.full((rows,), 1.0 / n, device="cuda"), dx, dw, ws)
    dgamma = torch.empty(cols, device="cuda")
    nws = torch.empty(M.moe_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    M.moe_norm_backward(M.MOE_NORM_RMS, dx, h, gamma, None, rstd, None, dh, dgamma, None, nws)
    out = torch.empty_like(w)
    ows = torch.empty(M.moe_orthogonalize_workspace_bytes(1, vocab, cols), dtype=torch.uint8, device="cuda")
    M.moe_orthogonalize(dw, None, 0.0, False, 5, 1e-7, 1.0, out, ows)
    torch.cuda.synchronize()
    # the whole step in 64 bits: the chain's roundings are bf16's, a few of them in a row
    s = to_f64(h)
    ry, _, rr = U.norm_forward("rms", s, to_f64(gamma), None, 1e-6)
    yy, wv = y.cpu().numpy(), to_f64(w)
    rloss, rlse = O.forward(ry, wv, yy)
    rdx, rdw = O.backward(ry, wv, yy, rlse, np.full(rows, 1.0 / n))
    rdh, rdg, _ = U.norm_backward("rms", rdx, s, to_f64(gamma), np.zeros(rows), rr)
    for name, got, want, steps in (("loss", loss, rloss, 1), ("dw", dw, rdw, 4), ("dh", dh, rdh, 5), ("dgamma", dgamma, rdg, 5)):
        off = np.linalg.norm(to_f64(got) - want) / np.linalg.norm(want)
        say(f"{name}: {off:.2e}")
        assert off <= steps * b16, name
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("dx,dw", [(True, True), (True, False), (False, True)])
def test_two_pieces(dx, dw):
    # 2^27 / 16448 rows is under 8192 columns a piece: two pieces, the second ragged and
    # shorter than the parts of dx's reduction would like
    c = Case(16400, 8, 8203, seed=11)
    c.forward()
    c.backward(dx, dw)
    torch.cuda.synchronize()
    c.check_backward(dx, dw)
    c.check_bands()


@pytest.mark.parametrize("rows,cols,vocab", [(400, 64, 3), (90, 256, 2), (600, 72, 130)])
def test_many_rows_with_one_target(rows, cols, vocab):
    c = Case(rows, cols, vocab, ignored=0.1, seed=12)
    c.y[c.y >= 0] = vocab - 1
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    c.check_forward()
    c.check_backward()
    c.check_bands()


@pytest.mark.parametrize("rows,cols,vocab", [(1, 512, 3000), (6, 256, 2000), (70, 384, 5000), (300, 512, 4000)])
def test_target_entries_are_held_finer(rows, cols, vocab):
    # rows of nearly uniform probabilities: the target's entry is all but the whole
    # gradient, and held in 16 bits.  What is left is the outputs' own rounding, b / sqrt 3
    # of a value at most on average, and that of entries whose squares sum to 1 / vocab
    # of the target's
    for seed in range(4):
        c = Case(rows, cols, vocab, ignored=0.0, seed=20 + seed, scale=0.05)
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        x, w, y = to_f64(c.x), to_f64(c.w), c.y.cpu().numpy()
        dx, dw = O.backward(x, w, y, to_f64(c.lse), to_f64(c.g))
        for got, want in ((c.dx, dx), (c.dw, dw)):
            off = np.linalg.norm(to_f64(got) - want) / np.linalg.norm(want)
            assert off <= b16 / 3 ** 0.5 * (1 + 4 / vocab ** 0.5), (seed, off)


def test_a_larger_batch_s_workspace():
    c = Case(40, 128, 3000, seed=13)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    want = [t.clone() for t in c.guards]
    c.work = torch.full((M.moe_head_loss_workspace_bytes(700, 128, 3000),), 255, dtype=torch.uint8, device="cuda")
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, c.guards))


@pytest.mark.parametrize("rows,cols,vocab", [(97, 264, 40), (1500, 200, 300), (900, 1000, 513), (1024, 4096, 4096)])
def test_a_few_targets_for_most_rows(rows, cols, vocab):
    """lists of targets longer than one stage of the reduction, in both tiles' columns"""
    c = Case(rows, cols, vocab, seed=21)
    rng = np.random.default_rng(22)
    few = rng.choice(vocab, 5, replace=False)
    y = c.y.cpu().numpy()
    often = rng.random(rows) < 0.85
    y[often] = few[rng.integers(0, 5, int(often.sum()))]
    c.y = torch.from_numpy(y).cuda()
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    c.check_bands()
