"""Refusals of moe_linear_lora_i8 and moe_logprobs (no GPU needed: every path returns before a HIP
call), and pins of their 64-bit forms."""
import ctypes

import numpy as np
import pytest
import torch

import bit_quantized_grouped_amd as bq
from oracle import serve_oracle

P = ctypes.c_void_p
F = P(0x10000)        # never dereferenced: validation fails first
ODD = P(0x10002)
NULL, SHAPE, ALIGN, WS = bq.MOE_ERR_NULL, bq.MOE_ERR_SHAPE, bq.MOE_ERR_ALIGN, bq.MOE_ERR_WORKSPACE
BIG = 1 << 40


def adapters(a=F, b=F, s=F, n=4, rank=16):
    return bq.MoeAdapters(a and a.value, b and b.value, s and s.value, n, rank)


def lora(a=F, s=F, M=4, K=128, w="ok", N=32, ad="ok", of=F, out=F, ws=F, wsb=BIG):
    w = bq.MoeI8Mat(F.value, F.value, 0) if w == "ok" else w
    ad = adapters() if ad == "ok" else ad
    return bq.lib().moe_linear_lora_i8(a, s, M, K, None if w is None else ctypes.byref(w), N,
                                       None if ad is None else ctypes.byref(ad), of, out, ws, wsb, None)


@pytest.mark.parametrize("kw,st", [
    (dict(M=0), SHAPE), (dict(N=0), SHAPE), (dict(K=96), SHAPE), (dict(K=131072), SHAPE), (dict(M=1 << 24), SHAPE),
    (dict(ad=None), NULL), (dict(ad=adapters(rank=0)), SHAPE), (dict(ad=adapters(rank=12)), SHAPE),
    (dict(ad=adapters(rank=136)), SHAPE), (dict(ad=adapters(rank=-8)), SHAPE), (dict(ad=adapters(n=0)), SHAPE),
    (dict(ad=adapters(n=-1)), SHAPE), (dict(ad=adapters(a=None)), NULL), (dict(ad=adapters(b=None)), NULL),
    (dict(ad=adapters(s=None)), NULL), (dict(ad=adapters(a=ODD)), ALIGN), (dict(ad=adapters(b=ODD)), ALIGN),
    (dict(ad=adapters(s=ODD)), ALIGN), (dict(a=None), NULL), (dict(s=None), NULL), (dict(w=None), NULL),
    (dict(of=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL), (dict(a=ODD), ALIGN), (dict(of=ODD), ALIGN),
    (dict(out=ODD), ALIGN), (dict(ws=P(0x10080)), ALIGN), (dict(wsb=64), WS), (dict(w=bq.MoeI8Mat(F.value, F.value, 2)), SHAPE)])
def test_lora_refusals(kw, st):
    assert lora(**kw) == st


def logprobs(z=F, dtype=0, ld=1000, t=F, T=4, V=1000, n=5, lp=F, ent=F, ti=F, tl=F, ws=F, wsb=BIG):
    return bq.lib().moe_logprobs(z, dtype, ld, t, T, V, n, lp, ent, ti, tl, ws, wsb, None)


@pytest.mark.parametrize("kw,st", [
    (dict(T=0), SHAPE), (dict(V=0), SHAPE), (dict(n=-1), SHAPE), (dict(n=65), SHAPE), (dict(V=4, ld=4), SHAPE),
    (dict(ld=999), SHAPE), (dict(ld=-5), SHAPE), (dict(ld=1 << 40), SHAPE), (dict(dtype=2), SHAPE), (dict(dtype=-1), SHAPE),
    (dict(n=0), SHAPE), (dict(ti=None, tl=None), SHAPE), (dict(z=None), NULL), (dict(t=None), NULL), (dict(lp=None), NULL),
    (dict(t=None, lp=None, ent=None, ti=None, tl=None, n=0), NULL), (dict(z=P(0x10001)), ALIGN), (dict(z=ODD, dtype=1), ALIGN),
    (dict(t=ODD), ALIGN), (dict(lp=ODD), ALIGN), (dict(ent=ODD), ALIGN), (dict(ti=ODD), ALIGN), (dict(tl=ODD), ALIGN),
    (dict(V=100000, ld=100000, ws=None), NULL), (dict(V=100000, ld=100000, wsb=8), WS),
    (dict(V=100000, ld=100000, ws=P(0x10080)), ALIGN)])
def test_logprobs_refusals(kw, st):
    assert logprobs(**kw) == st


def test_workspace_sizes():
    assert bq.linear_lora_i8_workspace_bytes(10, 64, 128, 16) >= 10 * 16 * 4
    assert bq.linear_lora_i8_workspace_bytes(10, 64, 128, 12) == 0 and bq.linear_lora_i8_workspace_bytes(0, 64, 128, 16) == 0
    assert bq.logprobs_workspace_bytes(1, 100000, 5) > 0 and bq.logprobs_workspace_bytes(5000, 100000, 5) == 0
    assert bq.logprobs_workspace_bytes(1, 100000, 65) == 0 and bq.logprobs_workspace_bytes(0, 100, 1) == 0


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("args,error", [
    ((bf(2, 16, 64).float(), bf(2, 32, 16), torch.zeros(2)), TypeError), ((bf(16, 64), bf(2, 32, 16), torch.zeros(2)), ValueError),
    ((bf(2, 16, 64), bf(3, 32, 16), torch.zeros(2)), ValueError), ((bf(2, 16, 64), bf(2, 32, 8), torch.zeros(2)), ValueError),
    ((bf(2, 16, 64), bf(2, 32, 16), torch.zeros(3)), ValueError), ((bf(2, 12, 64), bf(2, 32, 12), torch.zeros(2)), ValueError),
    ((bf(2, 136, 64), bf(2, 32, 136), torch.zeros(2)), ValueError), ((bf(0, 16, 64), bf(0, 32, 16), torch.zeros(0)), ValueError),
    ((bf(2, 64, 16).transpose(1, 2), bf(2, 32, 16), torch.zeros(2)), ValueError),
    ((bf(2, 16, 64), bf(2, 32, 16), torch.zeros(2, dtype=torch.float64)), TypeError)])
def test_adapter_sets_are_checked(args, error):
    with pytest.raises(error):
        bq.DeviceAdapters(*args)


def test_an_adapter_sets_tensors_are_fixed():
    ad = bq.DeviceAdapters(bf(2, 16, 64), bf(2, 32, 16), torch.zeros(2))
    with pytest.raises(AttributeError):
        ad.a = bf(2, 16, 64)


@pytest.mark.parametrize("part", ["a", "b", "scales"])
def test_adapters_that_moved_are_refused(part):
    """A tensor whose memory was exchanged in place: the call would read the old one."""
    ad = bq.DeviceAdapters(bf(2, 16, 64), bf(2, 32, 16), torch.zeros(2))
    args = dict(a=torch.zeros((3, 64), dtype=torch.int8), a_scale=torch.zeros(3),
                w=bq.DeviceI8Mat(torch.zeros((1, 32, 64), dtype=torch.int8), torch.zeros((1, 32))), adapters=ad,
                adapter=torch.zeros(3, dtype=torch.int32), out=bf(3, 32), ws=torch.zeros(1 << 12, dtype=torch.uint8))
    with pytest.raises(ValueError, match="device tensors"):
        bq.moe_linear_lora_i8(**args)
    t = getattr(ad, part)
    t.set_(t.clone())
    with pytest.raises(ValueError, match="lies elsewhere"):
        bq.moe_linear_lora_i8(**args)


@pytest.mark.parametrize("change,error", [
    (dict(a=torch.zeros((3, 64))), TypeError), (dict(a=torch.zeros((3, 128), dtype=torch.int8)), ValueError),
    (dict(a_scale=torch.zeros(4)), ValueError), (dict(w=None), TypeError), (dict(adapters=None), TypeError),
    (dict(adapters=bq.DeviceAdapters(bf(2, 16, 64), bf(2, 48, 16), torch.zeros(2))), ValueError),
    (dict(adapter=torch.zeros(3, dtype=torch.int64)), TypeError), (dict(adapter=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(out=bf(3, 31)), ValueError), (dict(ws=None), TypeError), ({}, ValueError)])   # the last: tensors on the CPU
def test_lora_binding_refusals(change, error):
    args = dict(a=torch.zeros((3, 64), dtype=torch.int8), a_scale=torch.zeros(3),
                w=bq.DeviceI8Mat(torch.zeros((1, 32, 64), dtype=torch.int8), torch.zeros((1, 32))),
                adapters=bq.DeviceAdapters(bf(2, 16, 64), bf(2, 32, 16), torch.zeros(2)),
                adapter=torch.zeros(3, dtype=torch.int32), out=bf(3, 32), ws=torch.zeros(1 << 12, dtype=torch.uint8))
    with pytest.raises(error):
        bq.moe_linear_lora_i8(**dict(args, **change))


I32 = torch.int32


@pytest.mark.parametrize("kw,error", [
    (dict(logits=torch.zeros(5, 100, dtype=torch.float16)), TypeError), (dict(logits=torch.zeros(100)), ValueError),
    (dict(logits=torch.zeros(100, 5).t()), ValueError), (dict(logits=torch.zeros(1, 100).expand(5, 100)), ValueError),
    (dict(logits=torch.zeros(5, 200)[:, ::2]), ValueError), (dict(targets=None), ValueError), (dict(logprob=None), ValueError),
    (dict(targets=torch.zeros(5, dtype=torch.int64)), TypeError), (dict(targets=torch.zeros(4, dtype=I32)), ValueError),
    (dict(entropy=torch.zeros(5, 1)), ValueError), (dict(top_idx=torch.zeros(5, 3)), TypeError),
    (dict(top_idx=torch.zeros((5, 0), dtype=I32)), ValueError), (dict(top_idx=torch.zeros(5, dtype=I32)), ValueError),
    (dict(top_idx=torch.zeros((5, 3), dtype=I32), top_logprob=torch.zeros(5, 4)), ValueError),
    (dict(targets=None, logprob=None, entropy=None), ValueError), (dict(ws=torch.zeros(4, 4).t()), ValueError), ({}, ValueError)])
def test_logprobs_binding_refusals(kw, error):
    args = dict(logits=torch.zeros(5, 100), targets=torch.zeros(5, dtype=I32), logprob=torch.zeros(5), entropy=torch.zeros(5))
    with pytest.raises(error):
        bq.moe_logprobs(**dict(args, **kw))


def test_oracle_of_log_probabilities():
    """Closed forms: equal logits, two tokens, a mask that leaves one token, an empty row."""
    ninf = -np.inf
    z = np.array([[1.0] * 4, [0.0, np.log(3.0), ninf, ninf], [ninf, 5.0, ninf, ninf], [ninf] * 4])
    lp, ent, idx, top = serve_oracle.logprobs(z, np.array([2, 1, 1, 0]), 2)
    np.testing.assert_allclose(lp[:3], [-np.log(4), np.log(0.75), 0], atol=1e-15)
    np.testing.assert_allclose(ent, [np.log(4), np.log(4) - 0.75 * np.log(3), 0, 0], atol=1e-15)
    assert idx.tolist() == [[0, 1], [1, 0], [1, 0], [0, 1]] and lp[3] == ninf and (top[3] == ninf).all()


def test_oracle_of_adapters():
    """An adapter is the matrix scale * B A beside W: one product with the sum is the same."""
    g = np.random.default_rng(0)
    a, w = g.integers(-9, 9, (5, 64)), g.integers(-9, 9, (7, 64))
    A, B, s = g.normal(size=(2, 8, 64)), g.normal(size=(2, 7, 8)), np.array([0.5, -2.0])
    sa, sw, of = g.random(5), g.random(7), np.array([0, 1, -1, 2, 1])
    out, _ = serve_oracle.linear_lora(a, sa, w, sw, A, B, s, of)
    for m, j in enumerate(of):
        W = w * sw[:, None] + (s[j] * B[j] @ A[j] if j in (0, 1) else 0)
        np.testing.assert_allclose(out[m], sa[m] * W @ a[m], rtol=1e-12)
