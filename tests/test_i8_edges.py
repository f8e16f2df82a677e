"""Calls of the 8-bit layer object and binding that went wrong without an error, on the CPU (no GPU
needed: every path ends at the device check or before)."""
import weakref

import pytest
import torch

import bit_quantized_grouped_amd as bq

BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8
T, H, I, E, k = 8, 256, 128, 16, 2


def i8mat(n, N, K, device="cpu"):
    return bq.DeviceI8Mat(torch.zeros((n, N, K), dtype=I8, device=device), torch.zeros((n, N), device=device))


def layer(**kw):
    mats = [i8mat(E, I, H), i8mat(E, I, H), i8mat(E, H, I)] + [None] * 3
    return bq.MoeLayerI8(mats, H, I, 0, E, k, "cpu", **kw)


def block(la, width=H, T=T):
    return la.forward_block(torch.zeros((T, width), dtype=BF16), None, torch.zeros(width, dtype=BF16),
                            torch.zeros((E, width), dtype=BF16))


def test_a_block_of_another_width_leaves_no_buffers_behind():
    la = layer()
    with pytest.raises(ValueError, match="the layer is H=256"):
        block(la, width=320)
    with pytest.raises(ValueError, match="w_router: shape"):
        la.forward_block(torch.zeros((T, H), dtype=BF16), None, torch.zeros(H, dtype=BF16), torch.zeros((E + 1, H), dtype=BF16))
    with pytest.raises(ValueError, match="device tensors"):   # all of it fits: the CPU is refused last
        block(la)
    assert la.buffers(T)["sum"].shape == (T, H)


def test_buffers_cannot_be_replaced():
    """A call keeps their addresses: a replaced entry would leave it writing to freed memory."""
    la = layer()
    b = la.buffers(T)
    with pytest.raises(TypeError, match="item assignment"):
        b["expert_out"] = torch.zeros((T * k, H), dtype=BF16)
    assert dict(b).keys() == {"routing", "route_ws", "gemm_ws", "expert_out", "shared_out", "y"}
    assert la.buffers(T)["y"] is b["y"]


@pytest.mark.parametrize("make,name,value", [
    (lambda: i8mat(E, I, H), "codes", torch.zeros((E, I, H), dtype=I8)), (lambda: i8mat(E, I, H), "scales", torch.ones(E, I)),
    (lambda: i8mat(E, I, H), "layout", 1), (lambda: i8mat(E, I, H), "struct", None), (bq.ScoreRule, "scale", 2.0),
    (bq.ScoreRule, "renormalise", False), (bq.ScoreRule, "n_groups", 4)])
def test_what_a_struct_was_made_of_stays(make, name, value):
    """The C call sees the struct alone: a new attribute would be ignored, or leave a freed address."""
    obj = make()
    before = getattr(obj, name)
    with pytest.raises(AttributeError, match="is fixed"):
        setattr(obj, name, value)
    assert getattr(obj, name) is before
    obj.note = "gate of layer 3"   # one of the caller's own


def test_released_buffers_are_freed_and_made_anew():
    la = layer()
    refs = {t: weakref.ref(la.buffers(t)["expert_out"]) for t in (3, T, 20)}
    la.release(T)
    assert refs[T]() is None and refs[3]() is not None and refs[20]() is not None
    assert la.buffers(T)["y"].shape == (T, H)
    la.release(7)   # never made
    la.release()
    assert all(r() is None for r in refs.values()) and la.buffers(3)["y"].shape == (3, H)


def wide(rows, cols, dtype):
    return torch.empty((rows, cols), dtype=dtype, device="meta")


#: 2^32 and some: its low 32 bits are a valid size.
BIG = (1 << 32) + 64


@pytest.mark.parametrize("call", [
    lambda: bq.moe_dequant_i8_bf16(wide(1, BIG, I8), torch.zeros(1), wide(1, BIG, BF16)),
    lambda: bq.moe_quant_i8(wide(BIG, 64, BF16), wide(BIG, 64, I8), wide(1, BIG, F32)[0]),
    lambda: bq.moe_norm_i8(wide(BIG, 64, BF16), None, torch.zeros(64, dtype=BF16), 1e-6, y=wide(BIG, 64, BF16)),
    lambda: bq.moe_linear_i8(wide(BIG, 64, I8), wide(1, BIG, F32)[0], i8mat(1, 16, 64), wide(BIG, 16, BF16)),
    lambda: bq.moe_route_scored(wide(BIG, 1, F32), None, bq.ScoreRule(), 1, 32, None, torch.zeros(256)),
    lambda: i8mat(1, BIG, 64, "meta"),
    lambda: bq.moe_i8_prepack(*[torch.empty((1, 16, BIG), dtype=I8, device="meta")] * 2),
    lambda: bq.DeviceRouting(BIG, 1, 1, 32, "meta"), lambda: bq.DeviceRouting(1, BIG, 1, 32, "meta")])
def test_sizes_past_32_bits_are_refused(call):
    """ctypes would pass their low 32 bits, and the call work on a part of its tensors."""
    with pytest.raises(ValueError, match="32"):
        call()


@pytest.mark.parametrize("K", [96, 16448])
def test_rows_that_cannot_be_quantised_are_named(K):
    """Before anything is allocated or enqueued: a matrix of E = 16 experts of N = 64."""
    w = torch.empty((E, 64, K), dtype=BF16)
    with pytest.raises(ValueError, match=f"K = {K}, expected a multiple of 64 up to 16384"):
        bq.DeviceI8Mat.from_bf16(w)
    with pytest.raises(ValueError, match=f"K = {K}"):
        bq.MoeLayerI8.from_bf16([w] * 3 + [None] * 3, K, 64, 0, E, k, "cpu")


@pytest.mark.parametrize("x,x_scale,logits,msg", [
    (torch.zeros((T, H + 64), dtype=I8), torch.zeros(T), torch.zeros(T, E), "the layer is H=256"),
    (torch.zeros((T, H)), torch.zeros(T), torch.zeros(T, E), "x: dtype"),
    (torch.zeros((T, H), dtype=I8), torch.zeros(T + 1), torch.zeros(T, E), "x_scale: shape"),
    (torch.zeros((T, H), dtype=I8), torch.zeros(T), torch.zeros(T, E + 1), "logits: shape")])
def test_a_refused_forward_keeps_no_buffers(x, x_scale, logits, msg):
    la = layer()
    with pytest.raises((TypeError, ValueError), match=msg):
        la.forward(x, x_scale, logits)
    assert not la._bufs
