"""GPU parity of the 4-bit-weight path (quantisation, packing, the grouped
products, the layer that runs on them) against the fp64 oracle, through the C ABI.

Codes and scales are decisions taken in the kernel's precision: bit for bit.

Tolerance of the products.  u = 2^-24 is half a step of fp32, b = 2^-8 of bf16.
Per group of G columns the accumulator takes 8 MFMAs at most, half with products
-136 a and half with (128 + code) a, code <= 15: products of magnitude at most
143 |a| each, exact, added in at most 8 levels an MFMA (32 products and the
accumulator): 72 roundings of a sum that 279 sum |a| bounds.  Then the scale's
product and the sum over groups (at most 64 here, and 4 waves' parts): 70 u of
the sum of the groups' magnitudes.  So y is off by at most
  d = u (72 * 279 sum_g |s_g| sum |a| + 70 sum_g |s_g y_g|),
down by d + b |y|; gate_up, with |silu'| <= 1.1 and |silu(g)| <= |g|, by
  1.1 |u| dg + |g| du + 2^-20 (1 + |g|) |h| + b |h| + dg du
(2^-20 (1 + |g|): the exponential's and the reciprocal's own errors).
"""
import numpy as np
import pytest
import torch

from mixture_experts_transformer_moe_amd import binding as M, configs
from mixture_experts_transformer_moe_amd.inputs import LayerInputs
from oracle import int4_oracle as I
from oracle import moe_oracle as O
from tests.gpu_common import StackedInputs, assert_close_rel, check_routing, out_tolerance, say, to_f64

pytestmark = pytest.mark.gpu

u32, b16 = 2.0 ** -24, 2.0 ** -8


def dev_bits(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).cuda()


class Case:
    """Random codes, scales and routing of one call; counts gives the rows of each expert."""

    def __init__(self, mode, T, D, F, Fs, group, counts, k, seed=0, scale_of=None, codes_of=None):
        rng = np.random.default_rng(seed)
        self.mode, self.group, self.E, self.k = mode, group, len(counts), k
        self.T, self.D, self.F, self.Fs, self.S = T, D, F, Fs, T * k
        assert sum(counts) <= self.S
        self.offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.sorted_token = rng.integers(0, T, self.S).astype(np.int32)
        K, N = (D, 2 * F) if mode == "gate_up" else (F, D)
        Ks, Ns = (D, 2 * Fs) if mode == "gate_up" else (Fs, D)
        code = codes_of or (lambda r, s: r.integers(-8, 8, s))
        scale = scale_of or (lambda r, s: 0.01 * np.exp(r.normal(size=s)))
        self.w, self.s = code(rng, (self.E, N, K)).astype(np.int8), bf16(scale(rng, (self.E, N, K // group)))
        self.ws = code(rng, (1, Ns, Ks)).astype(np.int8) if Fs else None
        self.ss = bf16(scale(rng, (1, Ns, Ks // group))) if Fs else None
        n_in = T * D if mode == "gate_up" else self.S * F + T * Fs
        self.a = bf16(rng.normal(size=n_in))
        self.shape = M.moe_shape(T, D, self.E, k, F, Fs, 1.0, M.MOE_BF16)
        n_out = self.S * F + T * Fs if mode == "gate_up" else self.S * D
        self.out = torch.full((n_out,), 7.0, dtype=torch.bfloat16, device="cuda")
        self.out_shared = torch.full((T * D,), 7.0, dtype=torch.bfloat16, device="cuda")
        self.pw = M.pack_int4(torch.from_numpy(I.two_a_byte(self.w)).cuda())
        self.pws = M.pack_int4(torch.from_numpy(I.two_a_byte(self.ws)).cuda()) if Fs else None
        self.off, self.tok = torch.from_numpy(self.offsets).cuda(), torch.from_numpy(self.sorted_token).cuda()
        self.x_perm = None

    def run(self, stream=None):
        if self.mode == "gate_up":
            M.moe_grouped_gate_up_int4(self.shape, self.group, self.x_perm, self.tok, self.a, self.off, self.pw, self.s,
                                       self.pws, self.ss, self.out, stream)
        else:
            M.moe_grouped_down_int4(self.shape, self.group, self.a, self.off, self.pw, self.s, self.pws, self.ss,
                                    self.out, self.out_shared if self.Fs else None, stream)

    def expected(self, rows, codes, scales):
        """(value, bound) of a product with one matrix [N, K]."""
        s = np.asarray(scales, np.float64)
        g = self.group
        a = rows.reshape(rows.shape[0], -1, g)
        c = codes.astype(np.float64).reshape(codes.shape[0], -1, g)
        y = np.zeros((rows.shape[0], codes.shape[0]))
        mag, tot = np.zeros_like(y), np.zeros_like(y)
        for i in range(a.shape[1]):
            part = (a[:, i] @ c[:, i].T) * s[:, i]
            y += part
            tot += np.abs(part)
            mag += np.abs(a[:, i]).sum(1)[:, None] * np.abs(s[:, i])
        d = u32 * (72 * 279 * mag + 70 * tot)
        if self.mode == "down":
            return y, d + b16 * np.abs(y)
        n = y.shape[1] // 2
        gate, up, dg, du = y[:, :n], y[:, n:], d[:, :n], d[:, n:]
        h = gate / (1 + np.exp(-gate)) * up
        return h, 1.1 * np.abs(up) * dg + np.abs(gate) * du + dg * du + (2.0 ** -20 * (1 + np.abs(gate)) + b16) * np.abs(h)

    def check(self, only=None):
        got = to_f64(self.out)
        a = to_f64(self.a)
        s = to_f64(self.s)
        width = self.F if self.mode == "gate_up" else self.D
        routed = got[: self.S * width].reshape(self.S, width)
        for e in range(self.E) if only is None else only:
            lo, hi = self.offsets[e], self.offsets[e + 1]
            if hi == lo:
                continue
            if self.mode == "gate_up":
                rows = a.reshape(self.T, self.D)[self.sorted_token[lo:hi]]
            else:
                rows = a[: self.S * self.F].reshape(self.S, self.F)[lo:hi]
            want, tol = self.expected(rows, self.w[e], s[e])
            bad = np.abs(routed[lo:hi] - want) > tol
            assert not bad.any(), f"expert {e}: {bad.sum()} of {bad.size} off, worst {(np.abs(routed[lo:hi] - want) / tol).max():.2f}"
        # rows behind the last routed one stay as they were
        assert (routed[self.offsets[-1]:] == 7.0).all()
        if self.Fs:
            if self.mode == "gate_up":
                rows, gs = a.reshape(self.T, self.D), got[self.S * width:].reshape(self.T, self.Fs)
            else:
                rows, gs = a[self.S * self.F:].reshape(self.T, self.Fs), to_f64(self.out_shared).reshape(self.T, self.D)
            want, tol = self.expected(rows, self.ws[0], to_f64(self.ss)[0])
            assert (np.abs(gs - want) <= tol).all(), "shared expert"


def counts_of(T, k, E, seed, kind):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return [0] * (E - 1) + [T * k]
    if kind == "masked":
        return list(rng.multinomial(T * k // 2, np.ones(E) / E))
    p = np.ones(E) if kind == "even" else 1.0 / np.arange(1, E + 1) ** 1.5
    return list(rng.multinomial(T * k, p / p.sum()))


# (T, k, E, D, F, Fs, counts)
SIZES = [(1, 1, 1, 256, 256, 0, "even"), (1, 4, 16, 512, 256, 256, "skew"), (3, 2, 8, 256, 768, 0, "masked"),
         (15, 1, 3, 768, 256, 512, "one"), (16, 2, 4, 1280, 512, 0, "even"), (17, 3, 5, 256, 512, 256, "skew"),
         (33, 1, 2, 2048, 256, 0, "one"), (70, 2, 70, 512, 512, 768, "skew"), (130, 2, 3, 256, 256, 256, "even"),
         (257, 1, 2, 512, 256, 256, "one"), (300, 4, 7, 256, 512, 0, "masked"), (600, 3, 4, 512, 256, 256, "skew"),
         (40, 16, 256, 256, 256, 256, "even"), (2, 1, 2, 4096, 1024, 1024, "even"), (700, 4, 5, 768, 1280, 256, "even")]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("mode", ["gate_up", "down"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_products(mode, group, size):
    T, k, E, D, F, Fs, kind = size
    say(f"int4 {mode} {size} group {group}")
    c = Case(mode, T, D, F, Fs, group, counts_of(T, k, E, T + E, kind), k, seed=T)
    c.run()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("mode", ["gate_up", "down"])
def test_extreme_codes_and_scales(mode):
    # all codes -8 (and 7), scales zero, negative, tiny and large
    pick = lambda r, s: r.choice([0.0, -0.01, 0.02, 2.0 ** -40, 8.0], s)  # noqa: E731
    for value in (-8, 7, 0):
        say(f"int4 {mode} codes {value}")
        c = Case(mode, 20, 512, 512, 256, 64, [5, 0, 20, 15], 2, seed=value + 9, scale_of=pick,
                 codes_of=lambda r, s: np.full(s, value))
        c.run()
        torch.cuda.synchronize()
        c.check()


def test_x_perm_equals_gather():
    c = Case("gate_up", 50, 512, 256, 256, 32, counts_of(50, 4, 9, 3, "skew"), 4, seed=5)
    c.run()
    first = c.out.clone()
    c.x_perm = c.a.view(50, 512)[c.tok.long()].contiguous()
    c.out.fill_(7.0)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)
    c.check()


@pytest.mark.parametrize("T", [4, 200])
def test_bad_tokens_stay_alone(T):
    # a token of NaN and one of infinities: their own rows alone change
    c = Case("gate_up", T, 256, 256, 256, 32, counts_of(T, 2, 4, 1, "even"), 2, seed=6)
    c.run()
    clean = c.out.clone()
    x = c.a.view(T, 256)
    x[1], x[2] = float("nan"), float("inf")
    c.out.fill_(7.0)
    c.run()
    torch.cuda.synchronize()
    routed, before = c.out[: c.S * 256].view(c.S, 256), clean[: c.S * 256].view(c.S, 256)
    hit = (c.tok == 1) | (c.tok == 2)
    assert torch.equal(routed[~hit], before[~hit])
    assert bool(torch.isnan(routed[c.tok == 1]).all()) and not bool(torch.isfinite(routed[c.tok == 2]).any())
    shared, before = c.out[c.S * 256:].view(T, 256), clean[c.S * 256:].view(T, 256)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[1:3] = False
    assert torch.equal(shared[keep], before[keep])


def test_offsets_out_of_range_stay_in_bounds():
    # a table that is no permutation's: rows outside [0, S) are never touched
    c = Case("down", 6, 256, 256, 0, 32, [2, 3, 1], 1, seed=2)
    c.off.copy_(torch.tensor([0, -5, 4, 1000], dtype=torch.int32))
    guard = torch.full((c.out.numel() + 2048,), 7.0, dtype=torch.bfloat16, device="cuda")
    c.out = guard[1024:-1024]
    c.run()
    torch.cuda.synchronize()
    assert (guard[:1024] == 7.0).all() and (guard[-1024:] == 7.0).all()


def test_repeats_bit_for_bit_on_streams_and_in_a_graph():
    a = Case("gate_up", 33, 1024, 256, 256, 64, counts_of(33, 4, 8, 1, "skew"), 4, seed=1)
    b = Case("down", 64, 256, 512, 256, 128, counts_of(64, 2, 6, 2, "even"), 2, seed=2)
    for c in (a, b):
        c.run()
    torch.cuda.synchronize()
    want = [a.out.clone(), b.out.clone(), b.out_shared.clone()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        a.out.zero_(), b.out.zero_(), b.out_shared.zero_()
        for st in streams:
            st.wait_stream(torch.cuda.current_stream())
        a.run(streams[0])
        with torch.cuda.stream(streams[1]):
            b.run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, (a.out, b.out, b.out_shared)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
        b.run()
    for i in range(3):
        a.out.zero_(), b.out.zero_(), b.out_shared.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, (a.out, b.out, b.out_shared))), i
        b.run()                                          # eager work between the replays
        torch.cuda.synchronize()
    # new inputs in the same buffers, and the routing with them
    x = Case("gate_up", 33, 1024, 256, 256, 64, counts_of(33, 4, 8, 7, "even"), 4, seed=8)
    for n in ("a", "off", "tok", "pw", "s", "pws", "ss"):
        getattr(a, n).copy_(getattr(x, n))
    g.replay()
    x.run()
    torch.cuda.synchronize()
    assert torch.equal(a.out, x.out)


def test_weights_past_32_bits():
    # 5 GB of codes: the last expert's lie past 2^32 bytes
    E, D, F = 40, 8192, 16384
    say("int4 gate_up, 5 GB of codes")
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 256, (E * 2 * F * D // 2,), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.full((E * 2 * F * D // 128,), 0.01, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(4, D, generator=g, device="cuda").to(torch.bfloat16)
    counts = torch.zeros(E, dtype=torch.int32)
    counts[0], counts[E - 1] = 1, 3
    off = torch.cat([torch.zeros(1, dtype=torch.int32), counts.cumsum(0).to(torch.int32)]).cuda()
    tok = torch.arange(4, dtype=torch.int32, device="cuda")
    h = torch.empty(4 * F, dtype=torch.bfloat16, device="cuda")
    M.moe_grouped_gate_up_int4(M.moe_shape(4, D, E, 1, F, 0, 1.0, M.MOE_BF16), 128, None, tok, x, off, codes, scales,
                               None, None, h)
    last = torch.empty(3 * F, dtype=torch.bfloat16, device="cuda")
    M.moe_grouped_gate_up_int4(M.moe_shape(3, D, 1, 1, F, 0, 1.0, M.MOE_BF16), 128, None, tok[:3], x[1:].contiguous(),
                               torch.tensor([0, 3], dtype=torch.int32, device="cuda"), codes[-F * D:].clone(),
                               scales[-2 * F * D // 128:].clone(), None, None, last)
    torch.cuda.synchronize()
    assert torch.isfinite(h).all()
    # another split of the reduction may round otherwise: two roundings of bf16 apart at most, and rarely
    a, b = h[F:].float(), last.float()
    assert ((a - b).abs() <= 2 * b16 * b.abs() + 1e-2 * b.abs().max() * b16).all()


# ------------------------------------------------------------------ load time

def test_quantise_is_bit_exact():
    rng = np.random.default_rng(5)
    count, rows, cols = 3, 48, 256
    w = rng.normal(0, 0.02, (count, rows, cols)).astype(np.float32)
    w[0, 3] = 0.0                                        # all-zero groups: scale 1, codes 0
    w[1, 7] *= 1e30
    w[1, 8] *= 1e-30
    w[1, 9] = 1e-40                                      # scales among the subnormals
    w[1, 10] = 9.2e-41                                   # the smallest subnormal: its seventh rounds to zero
    w[2, 10:13] = rng.choice(np.arange(-7, 7.5, 0.5), (3, cols))      # ties at scale 1
    w[2, 10:13, ::32] = 7.0
    bits = (w.view(np.uint32) >> 16).astype(np.uint16)
    for group in (32, 64, 128):
        codes, scales = M.quantize_int4(dev_bits(bits), group)
        torch.cuda.synchronize()
        ref_codes, ref_scales = I.quantize(bits, group)
        assert np.array_equal(scales.float().cpu().numpy(), ref_scales)
        assert np.array_equal(I.unpack(codes.cpu().numpy(), count, rows, cols), ref_codes)
        # the same codes through the other door
        packed = M.pack_int4(torch.from_numpy(I.two_a_byte(ref_codes)).cuda())
        assert torch.equal(packed, codes)


@pytest.mark.parametrize("count,rows,cols", [(1, 16, 128), (2, 32, 384), (5, 16, 256)])
def test_load_time_calls_write_their_outputs_only(count, rows, cols):
    rng = np.random.default_rng(9)
    bits = (rng.normal(0, 1, (count, rows, cols)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    n = count * rows * cols
    buf = torch.full((n // 2 + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    sc = torch.full((n // 32 + 4096,), -7.0, dtype=torch.bfloat16, device="cuda")
    M.moe_quantize_weights_int4(dev_bits(bits), buf[: n // 2], sc[: n // 32], count, rows, cols, 32)
    torch.cuda.synchronize()
    assert (buf[n // 2:] == 0xA5).all() and (sc[n // 32:] == -7.0).all()
    ref_codes, ref_scales = I.quantize(bits, 32)
    assert np.array_equal(I.unpack(buf[: n // 2].cpu().numpy(), count, rows, cols), ref_codes)
    assert np.array_equal(sc[: n // 32].float().cpu().numpy().reshape(ref_scales.shape), ref_scales)
    out = torch.full((n // 2 + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    M.moe_pack_weights_int4(torch.from_numpy(I.two_a_byte(ref_codes)).cuda(), out[: n // 2], count, rows, cols)
    torch.cuda.synchronize()
    assert (out[n // 2:] == 0xA5).all() and torch.equal(out[: n // 2], buf[: n // 2])


# ------------------------------------------------------------------ the layer

SMALL = configs.variant(configs.XS2_T4096, name="small_int4_t300", T=300, D=256, E=16, k=4, F=256, Fs=256)


@pytest.mark.parametrize("case,group", [("small", 128), ("rows150_E32", 64), ("T1", 32), ("T33_wide_shared", 128)])
def test_layer(case, group):
    kw = {"small": {}, "rows150_E32": dict(T=600, E=32, k=8), "T1": dict(T=1, D=512),
          "T33_wide_shared": dict(T=33, Fs=512)}[case]
    s = configs.variant(SMALL, name=f"int4_{case}", **kw)
    inp = StackedInputs(LayerInputs(s))
    w = M.upload_weights(s, inp.w_router, inp.bias, inp.wgu, inp.wd, inp.shared(), "cuda", int4=group)
    x = M.to_device(inp.x, s, "cuda")
    b = M.alloc_buffers(s, with_x_perm=case != "rows150_E32")
    M.layer_forward(s, x, w, b)
    torch.cuda.synchronize()
    check_routing(s, inp, b)
    ref, _ = O.forward(I.Int4Weights(inp, group), s.alpha, s.k, logits32=b.logits.cpu().numpy())
    say(f"{s.name}: {assert_close_rel(to_f64(b.out), ref, out_tolerance(s), 'out (4-bit weights)'):.2e}")


def test_decode_workload():
    s = configs.DECODE_SKEW_T32
    inp = StackedInputs(LayerInputs(s))
    w = M.upload_weights(s, inp.w_router, inp.bias, inp.wgu, inp.wd, inp.shared(), "cuda", int4=128)
    b = M.alloc_buffers(s, with_x_perm=False)
    M.layer_forward(s, M.to_device(inp.x, s, "cuda"), w, b)
    torch.cuda.synchronize()
    ref, _ = O.forward(I.Int4Weights(inp, 128), s.alpha, s.k, logits32=b.logits.cpu().numpy())
    assert_close_rel(to_f64(b.out), ref, out_tolerance(s), "out (4-bit weights)")


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("mode", ["gate_up", "down"])
def test_row_blocks_of_every_size(mode, group):
    """experts' rows around whole row blocks, and each number of token blocks in one"""
    say(f"int4 {mode} row blocks, group {group}")
    counts = [1, 17, 33, 49, 65, 81, 97, 113, 128, 129, 145, 177, 209, 256, 257, 289, 385]
    T = sum(counts) + 3
    c = Case(mode, T, 256, 256, 256, group, counts, 1, seed=31)
    c.run()
    torch.cuda.synchronize()
    c.check()
