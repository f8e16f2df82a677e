"""Refusals of the 8-bit operators: the C calls' statuses and the binding's checks (no GPU
needed: every path returns before a HIP call)."""
import ctypes

import pytest
import torch

import bit_quantized_grouped_amd as bq

P = ctypes.c_void_p
F = P(0x10000)        # never dereferenced: validation fails first
ODD = P(0x10008)
NULL, SHAPE, ALIGN, WS = bq.MOE_ERR_NULL, bq.MOE_ERR_SHAPE, bq.MOE_ERR_ALIGN, bq.MOE_ERR_WORKSPACE


def norm(x=F, res=F, w=F, eps=1e-6, T=4, H=128, s=F, y=F, q=F, qs=F):
    return bq.lib().moe_norm_i8(x, res, w, eps, T, H, s, y, q, qs, None)


@pytest.mark.parametrize("kw,st", [
    (dict(T=0), SHAPE), (dict(H=0), SHAPE), (dict(H=96), SHAPE), (dict(H=16448), SHAPE),
    (dict(eps=0.0), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(eps=float("inf")), SHAPE), (dict(x=None), NULL), (dict(w=None), NULL),
    (dict(q=None), NULL), (dict(qs=None), NULL), (dict(s=None, y=None, q=None, qs=None), NULL),
    (dict(x=ODD), ALIGN), (dict(res=ODD), ALIGN), (dict(w=ODD), ALIGN), (dict(s=ODD), ALIGN),
    (dict(y=ODD), ALIGN), (dict(q=ODD), ALIGN), (dict(qs=P(0x10002)), ALIGN)])
def test_norm_refusals(kw, st):
    assert norm(**kw) == st


@pytest.mark.parametrize("args,st", [
    ((F, 0, 128, F, F), SHAPE), ((F, 4, 100, F, F), SHAPE), ((F, 4, 16448, F, F), SHAPE),
    ((None, 4, 128, F, F), NULL), ((F, 4, 128, None, F), NULL), ((F, 4, 128, F, None), NULL),
    ((ODD, 4, 128, F, F), ALIGN), ((F, 4, 128, ODD, F), ALIGN), ((F, 4, 128, F, P(0x10002)), ALIGN)])
def test_quant_refusals(args, st):
    assert bq.lib().moe_quant_i8(*args, None) == st


@pytest.mark.parametrize("args,st", [
    ((F, F, 0, 128, F), SHAPE), ((F, F, 4, 100, F), SHAPE), ((None, F, 4, 128, F), NULL),
    ((F, None, 4, 128, F), NULL), ((F, F, 4, 128, None), NULL), ((ODD, F, 4, 128, F), ALIGN),
    ((F, F, 4, 128, ODD), ALIGN)])
def test_dequant_refusals(args, st):
    assert bq.lib().moe_dequant_i8_bf16(*args, None) == st


@pytest.mark.parametrize("args,st", [
    ((F, 0, 16, 64, P(0x20000)), SHAPE), ((F, 1, 24, 64, P(0x20000)), SHAPE),
    ((F, 1, 16, 32, P(0x20000)), SHAPE), ((F, 1 << 20, 1 << 16, 64, P(0x20000)), SHAPE),
    ((None, 1, 16, 64, F), NULL), ((F, 1, 16, 64, F), NULL), ((ODD, 1, 16, 64, F), ALIGN)])
def test_prepack_refusals(args, st):
    assert bq.lib().moe_i8_prepack(*args, None) == st


def mat(codes=F, scales=F, layout=0):
    return bq.MoeI8Mat(codes and codes.value, scales and scales.value, layout)


def linear(a=F, s=F, M=4, K=128, w="ok", N=32, out=F, ws=F, wsb=1 << 40):
    w = mat() if w == "ok" else w
    return bq.lib().moe_linear_i8(a, s, M, K, None if w is None else ctypes.byref(w), N, out, ws, wsb,
                                  None)


@pytest.mark.parametrize("kw,st", [
    (dict(M=0), SHAPE), (dict(N=0), SHAPE), (dict(K=32), SHAPE), (dict(K=131072), SHAPE),
    (dict(M=1 << 24), SHAPE), (dict(N=1 << 24), SHAPE),
    (dict(a=None), NULL), (dict(s=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL),
    (dict(w=mat(codes=None)), NULL), (dict(w=mat(scales=None)), NULL), (dict(w=mat(codes=ODD)), ALIGN),
    (dict(w=mat(layout=2)), SHAPE), (dict(w=mat(layout=1), N=33), SHAPE), (dict(a=ODD), ALIGN),
    (dict(out=ODD), ALIGN)])
def test_linear_refusals(kw, st):
    assert linear(**kw) == st


def rule(**kw):
    return bq.ScoreRule(**kw).struct


def raw(**kw):
    r = rule()
    for n, v in kw.items():
        setattr(r, n, v)
    return r


def scored(lg=F, bias=F, r="ok", T=4, E=32, k=4, br=32, out="ok", ws=F, wsb=1 << 40):
    r = rule(n_groups=4, topk_groups=2) if r == "ok" else r
    out = bq.MoeRouting(*([F.value] * 9)) if out == "ok" else out
    return bq.lib().moe_route_scored(lg, bias, None if r is None else ctypes.byref(r), T, E, k, br,
                                     None if out is None else ctypes.byref(out), ws, wsb, None)


@pytest.mark.parametrize("kw,st", [
    (dict(T=0), SHAPE), (dict(E=1001), SHAPE), (dict(k=0), SHAPE), (dict(br=8), SHAPE),
    (dict(lg=None), NULL), (dict(r=None), NULL), (dict(out=None), NULL), (dict(T=20000, ws=None), NULL),
    (dict(r=raw(score=2)), SHAPE), (dict(r=raw(group_score=-1)), SHAPE), (dict(r=raw(renormalise=2)), SHAPE),
    (dict(r=raw(scale=float("nan"))), SHAPE), (dict(r=raw(scale=float("inf"))), SHAPE),
    (dict(r=raw(n_groups=0)), SHAPE), (dict(r=raw(n_groups=5, topk_groups=1)), SHAPE),
    (dict(r=raw(n_groups=128, topk_groups=1), E=128), SHAPE), (dict(r=raw(n_groups=4, topk_groups=0)), SHAPE),
    (dict(r=raw(n_groups=4, topk_groups=5)), SHAPE),
    (dict(r=raw(n_groups=32, topk_groups=32, group_score=1)), SHAPE),   # groups of one have no second best
    (dict(r=raw(n_groups=16, topk_groups=1)), SHAPE),                   # k = 4 of groups of two
    (dict(r=raw(), E=128, k=65), SHAPE),
    (dict(lg=P(0x10002)), ALIGN), (dict(bias=P(0x10002)), ALIGN), (dict(ws=P(0x10010)), ALIGN),
    (dict(T=20000, wsb=16), WS)])
def test_scored_routing_refusals(kw, st):
    assert scored(**kw) == st


def grouped(x=F, s=F, T=8, H=256, I=128, I_sh=128, E=16, k=2, br=32, r="ok", mats=None, eo=F, so=F,
            ws=F, wsb=1 << 40):
    r = bq.MoeRouting(*([F.value] * 9)) if r == "ok" else r
    mats = mats or [mat()] * 6
    args = [x, s, T, H, I, I_sh, E, k, br, None if r is None else ctypes.byref(r)]
    args += [None if m is None else ctypes.byref(m) for m in mats]
    return bq.lib().moe_grouped_gemm_i8(*args, eo, so, ws, wsb, None)


def but(i, m):
    return [m if j == i else mat() for j in range(6)]


@pytest.mark.parametrize("kw,st", [
    (dict(T=0), SHAPE), (dict(H=96), SHAPE), (dict(I=0), SHAPE), (dict(k=17), SHAPE), (dict(br=128), SHAPE),
    (dict(H=131072, T=1), SHAPE), (dict(H=65536, I=32768, T=1), SHAPE), (dict(x=None), NULL),
    (dict(s=None), NULL), (dict(r=None), NULL), (dict(eo=None), NULL), (dict(so=None), NULL),
    (dict(ws=None), NULL), (dict(mats=but(0, None)), NULL), (dict(mats=but(5, None)), NULL),
    (dict(mats=but(1, mat(layout=1))), SHAPE), (dict(mats=but(4, mat(layout=1))), SHAPE),
    (dict(mats=but(2, mat(codes=ODD))), ALIGN), (dict(I_sh=0), SHAPE), (dict(x=ODD), ALIGN),
    (dict(eo=ODD), ALIGN), (dict(so=ODD), ALIGN), (dict(ws=P(0x10010)), ALIGN), (dict(wsb=1024), WS)])
def test_grouped_refusals(kw, st):
    assert grouped(**kw) == st


def test_workspace_sizes():
    w = bq.gemm_i8_workspace_bytes
    assert w(512, 2048, 512, 512, 256, 8, 32) >= 5 * 512 * 9 * 512 + 4 * 512 * 9
    assert w(0, 2048, 512, 512, 256, 8, 32) == 0 and w(8, 131072, 64, 0, 4, 1, 32) == 0
    assert bq.linear_i8_workspace_bytes(0, 16, 64) == 0


def test_layer_refuses_a_bias_without_a_rule():
    r, m = bq.MoeRouting(*([F.value] * 9)), mat()
    args = [F, F, F, F, None, 8, 256, 128, 128, 16, 2, 32] + [ctypes.byref(m)] * 6
    args += [ctypes.byref(r), F, 1 << 30, F, F, F, 1 << 30, F, None]
    assert bq.lib().moe_layer_i8(*args) == SHAPE


# ---- the binding, on CPU tensors: mistakes are named before the device check ----

T, H, I, E, k = 8, 256, 128, 16, 2


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def i8(*s):
    return torch.zeros(s, dtype=torch.int8)


def f32(*s):
    return torch.zeros(s)


def i8mat(n, N, K):
    return bq.DeviceI8Mat(i8(n, N, K), f32(n, N))


@pytest.mark.parametrize("call,exc,msg", [
    (lambda: bq.moe_norm_i8(f32(T, H), None, bf(H), 1e-6, y=bf(T, H)), TypeError, "x: dtype"),
    (lambda: bq.moe_norm_i8(bf(T, H), None, bf(H + 64), 1e-6, y=bf(T, H)), ValueError, "weight: shape"),
    (lambda: bq.moe_norm_i8(bf(T, H), bf(1, H), bf(H), 1e-6, y=bf(T, H)), ValueError, "residual: shape"),
    (lambda: bq.moe_norm_i8(bf(T, H), bf(H, T).t(), bf(H), 1e-6, y=bf(T, H)), ValueError, "contiguous"),
    (lambda: bq.moe_norm_i8(bf(T, H), None, bf(H), 1e-6, q=i8(T, H)), ValueError, "both or neither"),
    (lambda: bq.moe_norm_i8(bf(T, H), None, bf(H), 1e-6), ValueError, "at least one"),
    (lambda: bq.moe_norm_i8(bf(T, H), None, bf(H), 1e-6, y=bf(T, H)), ValueError, "device tensors"),
    (lambda: bq.moe_quant_i8(bf(T, H), i8(T, H), f32(T + 1)), ValueError, "scale: shape"),
    (lambda: bq.moe_dequant_i8_bf16(i8(T, H), f32(T), bf(T, H + 64)), ValueError, "out: shape"),
    (lambda: bq.moe_linear_i8(i8(T, H), f32(T), i8mat(1, 32, H + 64), bf(T, 32)), ValueError, "w: codes"),
    (lambda: bq.moe_linear_i8(i8(T, H), f32(T), i8mat(2, 32, H), bf(T, 32)), ValueError, "w: codes"),
    (lambda: bq.moe_linear_i8(i8(T, H), f32(T, 1), i8mat(1, 32, H), bf(T, 32)), ValueError, "a_scale: shape"),
    (lambda: bq.moe_linear_i8(i8(T, H), f32(T), "w", bf(T, 32)), TypeError, "DeviceI8Mat"),
    (lambda: bq.DeviceI8Mat(i8(4, 32, 64), f32(4, 31)), ValueError, "scales: shape"),
    (lambda: bq.DeviceI8Mat(i8(32, 64), f32(32)), ValueError, "n_exp"),
    (lambda: bq.DeviceI8Mat(i8(4, 32, 64), f32(4, 32), 2), ValueError, "layout"),
    (lambda: bq.DeviceI8Mat(i8(4, 32, 64), f32(4, 32), 1).prepacked(), ValueError, "in tiles already"),
    (lambda: bq.ScoreRule(score="relu"), ValueError, "score"),
    (lambda: bq.ScoreRule(group_score="sum"), ValueError, "group_score"),
    (lambda: bq.moe_route_scored(f32(T, E), f32(E + 1), bq.ScoreRule(), k, 32,
                                 bq.DeviceRouting(T, E, k, 32, "cpu"), i8(256)), ValueError, "bias: shape"),
    (lambda: bq.moe_route_scored(f32(T, E), None, None, k, 32,
                                 bq.DeviceRouting(T, E, k, 32, "cpu"), i8(256)), TypeError, "ScoreRule"),
    (lambda: bq.moe_route_scored(f32(T, E), None, bq.ScoreRule(), k, 32,
                                 bq.DeviceRouting(T + 1, E, k, 32, "cpu"), i8(256)), ValueError, "built for"),
    (lambda: bq.MoeLayerI8([i8mat(E, I, H)] * 3 + [None] * 3, H, I, 0, E, k, "cpu"), ValueError, "down: codes"),
    (lambda: bq.MoeLayerI8([i8mat(E, I, H), i8mat(E, I, H), i8mat(E, H, I)] + [None] * 3, H, I, I, E, k, "cpu"),
     TypeError, "sh_gate"),
])
def test_binding_refusals(call, exc, msg):
    with pytest.raises(exc, match=msg):
        call()


def test_layer_buffers_must_match():
    mats = [i8mat(E, I, H), i8mat(E, I, H), i8mat(E, H, I)] + [None] * 3
    def call(x=i8(T, H), lg=f32(T, E), eo=bf(T * k, H), y=bf(T, H), bias=None, rule=None):
        bq.moe_layer_i8(x, f32(T), lg, bias, rule, I, 0, E, k, 32, bq.DeviceRouting(T, E, k, 32, "cpu"),
                        i8(256), *mats, eo, None, i8(256), y)
    for kw, msg in [(dict(lg=f32(T, E + 1)), "logits: shape"), (dict(eo=bf(T, H)), "expert_out: shape"),
                    (dict(y=bf(T, H + 64)), "y: shape"), (dict(bias=f32(E)), "needs a rule"),
                    (dict(), "device tensors")]:
        with pytest.raises(ValueError, match=msg):
            call(**kw)
