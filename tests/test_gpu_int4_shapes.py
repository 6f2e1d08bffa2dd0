"""The binding takes the 4-bit calls' tensors as the header has them, or with dimensions joined
(flat) or split (tokens as sequences); the same number of elements in another order is refused."""
import pytest
import torch

from mixture_experts_transformer_moe_amd import binding as M

pytestmark = pytest.mark.gpu

T, D, E, k, F, Fs, G = 6, 256, 4, 2, 512, 256, 32


def z(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt, device="cuda")


def gate_up_args():
    return dict(x_perm=None, sorted_token=z(T * k, dt=torch.int32), x=z(T, D), offsets=z(E + 1, dt=torch.int32),
                w_gate_up=z(E * F * D, dt=torch.uint8), w_gate_up_scale=z(E, 2 * F, D // G),
                ws_gate_up=z(Fs * D, dt=torch.uint8), ws_gate_up_scale=z(2 * Fs, D // G), h=z(T * k * F + T * Fs))


def down_args():
    return dict(h=z(T * k * F + T * Fs), offsets=z(E + 1, dt=torch.int32), w_down=z(E * D * F // 2, dt=torch.uint8),
                w_down_scale=z(E, D, F // G), ws_down=z(D * Fs // 2, dt=torch.uint8), ws_down_scale=z(D, Fs // G),
                y_perm=z(T * k, D), y_shared=z(T, D))


CALLS = [(M.moe_grouped_gate_up_int4, gate_up_args), (M.moe_grouped_down_int4, down_args)]


def call(fn, args):
    fn(M.moe_shape(T, D, E, k, F, Fs, 1.0, M.MOE_BF16), G, *args.values())
    torch.cuda.synchronize()


@pytest.mark.parametrize("fn,args", CALLS, ids=["gate_up", "down"])
def test_shapes_of_the_header_joined_and_split(fn, args):
    call(fn, args())
    for name, t in args().items():
        if t is None:
            continue
        ok = [t.reshape(-1), t.reshape(1, *t.shape)]
        if t.dim() > 1:
            ok += [t.reshape(2, t.shape[0] // 2, *t.shape[1:]), t.reshape(*t.shape[:-1], 2, -1)]
        if t.dim() == 3:
            ok += [t.reshape(-1, t.shape[-1]), t.reshape(t.shape[0], -1)]
        for other in ok:
            call(fn, {**args(), name: other})


@pytest.mark.parametrize("fn,args", CALLS, ids=["gate_up", "down"])
def test_other_orders_are_refused(fn, args):
    for name, t in args().items():
        if t is None or t.dim() == 1:
            continue
        bad = [t.transpose(-1, -2).contiguous()]
        if t.dim() == 3:
            bad.append(t.transpose(0, 1).contiguous())
        for other in bad:
            with pytest.raises(ValueError, match=name):
                call(fn, {**args(), name: other})


def test_load_time_calls():
    n = 2 * 32 * 256
    w, codes = z(2, 32, 256), z(2, 32, 128, dt=torch.uint8)
    packed, scales = z(n // 2, dt=torch.uint8), z(2, 32, 8)
    M.moe_quantize_weights_int4(w, packed, scales, 2, 32, 256, 32)
    M.moe_quantize_weights_int4(w.view(64, 256), packed, scales.view(64, 8), 2, 32, 256, 32)
    M.moe_pack_weights_int4(codes, packed, 2, 32, 256)
    torch.cuda.synchronize()
    for bad in ((z(2, 256, 32), packed, scales), (w, packed, z(2, 8, 32)), (w, packed, z(8, 2, 32))):
        with pytest.raises(ValueError):
            M.moe_quantize_weights_int4(*bad, 2, 32, 256, 32)
    with pytest.raises(ValueError, match="codes"):
        M.moe_pack_weights_int4(z(2, 128, 32, dt=torch.uint8), packed, 2, 32, 256)
