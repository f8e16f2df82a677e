"""Refusals of moe_decode_batch_q4 and MoeLayer.decode_batch (no GPU needed: every path returns
before a HIP call)."""
import ctypes

import pytest
import torch

import bit_quantized_grouped_amd as bq

P = ctypes.c_void_p
F = P(0x10000)        # never dereferenced: validation fails first
ODD = P(0x10002)
NULL, SHAPE, ALIGN, WS = bq.MOE_ERR_NULL, bq.MOE_ERR_SHAPE, bq.MOE_ERR_ALIGN, bq.MOE_ERR_WORKSPACE
DIMS = dict(T=8, H=256, I=128, I_sh=64, E=16, k=4)


def mat(codes=F, scales=F, biases=F, layout=0):
    return bq.MoeQ4Mat(*(p and p.value for p in (codes, scales, biases)), layout)


def call(x=F, lg=F, bias=None, rule=None, gate=None, idx=F, w=F, y=F, ws=F, wsb=1 << 40, mats=None, **dims):
    d = dict(DIMS, **dims)
    mats = mats or [mat()] * 3 + [mat() if d["I_sh"] else None] * 3
    refs = [None if m is None else ctypes.byref(m) for m in mats]
    return bq.lib().moe_decode_batch_q4(
        x, lg, bias, None if rule is None else ctypes.byref(rule.struct), gate, d["T"], d["H"], d["I"],
        d["I_sh"], d["E"], d["k"], *refs, idx, w, y, ws, wsb, None)


def with_mat(i, m):
    mats = [mat()] * 6
    mats[i] = m
    return mats


@pytest.mark.parametrize("kw,st", [
    (dict(T=0), SHAPE), (dict(T=65), SHAPE), (dict(H=96), SHAPE), (dict(I=0), SHAPE), (dict(I_sh=-64), SHAPE),
    (dict(H=1 << 24, I=64, I_sh=64), SHAPE),
    (dict(E=0), SHAPE), (dict(E=1001), SHAPE), (dict(k=17), SHAPE), (dict(k=0), SHAPE),
    (dict(k=65, E=100), SHAPE), (dict(x=None), NULL), (dict(lg=None), NULL), (dict(y=None), NULL),
    (dict(ws=None), NULL), (dict(idx=None), NULL), (dict(w=None), NULL), (dict(bias=F), SHAPE),
    (dict(x=ODD), ALIGN), (dict(y=ODD), ALIGN), (dict(lg=ODD), ALIGN), (dict(gate=ODD), ALIGN),
    (dict(idx=ODD), ALIGN), (dict(w=ODD), ALIGN), (dict(ws=P(0x10080)), ALIGN), (dict(wsb=100), WS),
    (dict(gate=F, I_sh=0), SHAPE), (dict(I_sh=0, mats=[mat()] * 6), SHAPE),
    (dict(mats=with_mat(0, None)), NULL), (dict(mats=with_mat(4, None)), NULL),
    (dict(mats=with_mat(1, mat(codes=None))), NULL), (dict(mats=with_mat(2, mat(scales=ODD, biases=P(1)))), ALIGN),
    (dict(mats=with_mat(1, mat(layout=1))), SHAPE), (dict(mats=with_mat(2, mat(layout=2))), SHAPE),
    (dict(mats=with_mat(0, mat(layout=3))), SHAPE),
    (dict(rule=bq.ScoreRule(n_groups=3)), SHAPE), (dict(rule=bq.ScoreRule(n_groups=8, topk_groups=1)), SHAPE),
    (dict(rule=bq.ScoreRule(scale=float("inf"))), SHAPE)])
def test_refusals(kw, st):
    assert call(**kw) == st


def test_workspace_size():
    size = bq.decode_batch_workspace_bytes
    assert size(8, 256, 128, 64, 16, 4) >= 8 * (4 * 128 + 64) * 4
    assert size(0, 256, 128, 64, 16, 4) == 0 and size(65, 256, 128, 64, 16, 4) == 0
    assert size(8, 256, 100, 64, 16, 4) == 0 and size(8, 256, 128, 64, 100, 65) == 0


def qmat(n_exp, N, K, layout=0):
    sb = layout == bq.LAYOUT_TILES_SB
    s = torch.zeros((n_exp, N, K // 64), dtype=torch.int32 if sb else torch.bfloat16)
    return bq.DeviceQMat(torch.zeros((n_exp, N, K // 8), dtype=torch.int32), s, None if sb else s.clone(), layout)


def layer(**kw):
    d = dict(H=128, I=64, I_sh=64, E=8, k=2, **kw)
    H, I, I_sh, E = d["H"], d["I"], d["I_sh"], d["E"]
    mats = [qmat(E, I, H), qmat(E, I, H), qmat(E, H, I), qmat(1, I_sh, H), qmat(1, I_sh, H), qmat(1, H, I_sh)]
    return bq.MoeLayer.from_device(mats, H, I, I_sh, E, d["k"], "cpu")


X, LG = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros((4, 8))


@pytest.mark.parametrize("args,kw,error", [
    ((X.float(), LG), {}, TypeError), ((X[0], LG), {}, ValueError), ((X[:0], LG[:0]), {}, ValueError),
    ((torch.zeros((65, 128), dtype=torch.bfloat16), torch.zeros((65, 8))), {}, ValueError),
    ((X[:, :64].contiguous(), LG), {}, ValueError), ((X, LG[:3]), {}, ValueError), ((X, LG.double()), {}, TypeError),
    ((torch.zeros((128, 4), dtype=torch.bfloat16).t(), LG), {}, ValueError), ((X, None), {}, TypeError),
    ((X, LG), dict(score_bias=torch.zeros(8)), ValueError), ((X, LG), dict(rule="softmax"), TypeError),
    ((X, LG), dict(rule=bq.ScoreRule(), score_bias=torch.zeros(7)), ValueError),
    ((X, LG), dict(shared_gate=torch.zeros(3)), ValueError), ((X, LG), dict(shared_gate=torch.zeros(4, 1)), ValueError),
    ((X, LG), {}, ValueError)])   # tensors on the CPU
def test_layer_object_refusals(args, kw, error):
    m = layer()
    with pytest.raises(error):
        m.decode_batch(*args, **kw)
    assert not m._batch_bufs


def test_matrix_sets_are_checked():
    m = layer()
    m.down = qmat(8, 64, 128)
    with pytest.raises(ValueError, match="down"):
        m.decode_batch(X, LG)
    m = layer()
    m.up.codes = m.up.codes.to(torch.int64)
    with pytest.raises(TypeError, match="up.codes"):
        m.decode_batch(X, LG)
    m = layer()
    m.up.codes = m.up.codes.clone()   # the struct holds the first tensor's address
    with pytest.raises(ValueError, match="another tensor"):
        m.decode_batch(X, LG)


def replaced(m, part):
    t = getattr(m.gate, part)
    setattr(m.gate, part, t + 1 if part == "layout" else t.clone())


def moved(m, part):
    getattr(m.down, part).set_(getattr(m.down, part).clone())   # the same tensor, elsewhere


@pytest.mark.parametrize("change,part,match", [
    (replaced, "codes", "gate.codes: another"), (replaced, "scales", "gate.scales: another"),
    (replaced, "biases", "gate.biases: another"), (replaced, "layout", "gate.layout: another"),
    (moved, "codes", "down.codes: another"), (moved, "biases", "down.biases: another")])
def test_matrix_sets_are_checked_again_when_they_change(change, part, match):
    """A set is checked at the object's first call; one whose tensors are replaced afterwards is
    refused as it is before it, and not used with the tensors of then."""
    m = layer()
    for _ in range(2):
        with pytest.raises(ValueError, match="device tensors"):   # the sets are as they should be
            m.decode_batch(X, LG)
    change(m, part)
    for _ in range(2):
        with pytest.raises(ValueError, match=match):
            m.decode_batch(X, LG)


def test_sizes_that_change_are_taken_up():
    """Matrix sets that no longer hold the layer's sizes are refused after its first call too."""
    for name, value in (("E", 16), ("I", 128), ("I_sh", 128), ("I_sh", 0)):
        m = layer()
        with pytest.raises(ValueError, match="device tensors"):
            m.decode_batch(X, LG)
        setattr(m, name, value)
        with pytest.raises(ValueError, match="do not hold|must be None"):
            m.decode_batch(X, torch.zeros((4, m.E)))


def test_binding_refusals():
    m = layer().weight_mats()
    ws, y = torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros_like(X)
    with pytest.raises(ValueError, match="both or neither"):
        bq.moe_decode_batch_q4(X, LG, None, None, None, 64, 64, 2, *m, y, ws, torch.zeros((4, 2), dtype=torch.int32))
    with pytest.raises(ValueError, match="must be None"):
        bq.moe_decode_batch_q4(X, LG, None, None, torch.zeros(4), 64, 0, 2, *m[:3], None, None, None, y, ws)
    with pytest.raises(ValueError, match="device tensors"):
        bq.moe_decode_batch_q4(X, LG, None, None, None, 64, 64, 2, *m, y, ws)


def test_release_without_buffers():
    m = layer()
    m.release()
    m.release(7)
    m._batch_bufs[4, (-1,)], m._batch_bufs[5, (-1,)], m._bufs[4] = {}, {}, {}
    m.release(4)
    assert list(m._batch_bufs) == [(5, (-1,))] and not m._bufs
    m.release()
    assert not m._batch_bufs
