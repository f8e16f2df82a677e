"""MoeLayer.decode_batch's buffers and matrix sets over its object's life, on the GPU."""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_amd as bq
import test_gpu_batch as tb
from gpu_cases import DEV, announce, require_gpu

pytestmark = pytest.mark.gpu


def test_release_gives_the_memory_back():
    require_gpu()
    announce("batch, release")
    H, I, I_sh, E, k = 1024, 512, 64, 64, 8
    g = np.random.default_rng(1)
    mats = tb.device_mats(tb.host_mats(g, E, H, I, I_sh), bq.LAYOUT_TILES_SB)
    layer = bq.MoeLayer.from_device(mats, H, I, I_sh, E, k, DEV)
    x, lg = tb.inputs(g, 64, H, E)
    run = lambda T, **kw: layer.decode_batch(x[:T], lg[:T], **kw)["y"].clone()  # noqa: E731
    want = {T: run(T) for T in (3, 20)}
    start = torch.cuda.memory_allocated()
    for T in range(50, 65):
        run(T)
    run(64, stream=torch.cuda.Stream())   # still on its way when the buffers go
    assert torch.cuda.memory_allocated() - start > 60_000_000
    for T in range(50, 65):
        layer.release(T)
    assert torch.cuda.memory_allocated() - start < 1_000_000
    assert torch.equal(run(20), want[20])   # kept
    layer.release()
    assert torch.cuda.memory_allocated() < start
    for T, w in want.items():
        assert torch.equal(run(T), w)
    tb.sync()


def test_sets_that_change_after_a_call():
    """A set with replaced codes is refused, and the layer goes on with a set made of them."""
    require_gpu()
    announce("batch, replaced codes")
    T, H, I, E, k = 4, 128, 64, 8, 2
    g = np.random.default_rng(8)
    a, b = (tb.device_mats(tb.host_mats(g, E, H, I, 0), bq.LAYOUT_TILES) for _ in range(2))
    x, lg = tb.inputs(g, T, H, E)
    layer = bq.MoeLayer.from_device(a, H, I, 0, E, k, DEV)
    first = layer.decode_batch(x, lg)["y"].clone()
    a[1].codes = b[1].codes
    with pytest.raises(ValueError, match="up.codes: another tensor"):
        layer.decode_batch(x, lg)
    layer.up = bq.DeviceQMat(b[1].codes, a[1].scales, a[1].biases, bq.LAYOUT_TILES)
    second = layer.decode_batch(x, lg)["y"].clone()
    layer.k = 3   # other buffers than for two a token
    third = layer.decode_batch(x, lg)
    want = bq.MoeLayer.from_device(layer.weight_mats(), H, I, 0, E, 3, DEV).decode_batch(x, lg)["y"]
    tb.sync()
    assert third["topk_idx"].shape == (T, 3) and torch.equal(third["y"], want)
    assert not torch.equal(first, second)
