"""The 8-bit operators on the GPU at the edges of what they take.

Tolerances are those of test_gpu_i8.py, whose helpers and 64-bit forms these tests use.
"""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_amd as bq
from gpu_cases import DEV, announce, require_gpu
from oracle import i8_oracle as ref
from test_gpu_i8 import EPS, check_norm, dev, f64, norm_inputs, sync, within

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


# ---- NaN and infinities ----

# a wave a row, four waves, eight of one piece, eight of two, sixteen
@pytest.mark.parametrize("H", [64, 1024, 2048, 4096, 7168, 8256])
def test_norm_of_rows_with_nan_and_infinities(H):
    """Such a row's scale is NaN (infinite where only the weight is), its codes 0; the other rows
    are what they are without it."""
    require_gpu()
    announce(f"norm with NaN H={H}")
    T = 7
    x, r, w = norm_inputs(T, H, H)
    x[1, H - 3], r[2, 0], x[4, 5], r[5, H // 2] = NAN, NAN, INF, -INF
    s, y = torch.empty_like(x), torch.empty_like(x)
    q, qs = torch.full((T, H), 5, dtype=torch.int8, device=DEV), torch.zeros(T, device=DEV)
    bq.moe_norm_i8(x, r, w, EPS, s, y, q, qs)
    sync()
    bad, good = [1, 2, 4, 5], [0, 3, 6]
    assert qs[bad].isnan().all() and not q[bad].any()
    same = lambda a, b: torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())  # noqa: E731
    assert y[[1, 2]].isnan().all() and same(s, (x.float() + r.float()).bfloat16())
    assert torch.equal(y.isnan().sum(1)[[4, 5]].cpu(), torch.tensor([1, 1]))   # v / sqrt(inf) is 0 beside inf / inf
    check_norm(x[good], r[good], w, s[good], y[good], q[good], qs[good])
    for bad_weight, top in ((NAN, NAN), (INF, INF)):
        w[7] = bad_weight
        bq.moe_norm_i8(x[good], r[good], w, EPS, q=q[:3], q_scale=qs[:3])
        sync()
        assert not q[:3].any() and same(qs[:3], torch.full((3,), top, device=DEV))


@pytest.mark.parametrize("K", [64, 1024, 1088, 4096, 8192, 8256])
def test_quant_of_rows_with_nan_and_infinities(K):
    require_gpu()
    announce(f"quant with NaN K={K}")
    x = dev(np.random.default_rng(K).normal(size=(6, K)), torch.bfloat16)
    x[0, K - 1], x[2], x[3, 9], x[5, 1], x[5, 2] = NAN, NAN, -INF, INF, NAN
    q, s = torch.full((6, K), 5, dtype=torch.int8, device=DEV), torch.zeros(6, device=DEV)
    back = torch.zeros_like(x)
    bq.moe_quant_i8(x, q, s)
    bq.moe_dequant_i8_bf16(q, s, back)
    sync()
    bad, good = [0, 2, 3, 5], [1, 4]
    assert s[[0, 2, 5]].isnan().all() and float(s[3]) == INF and not q[bad].any() and back[bad].isnan().all()
    _, scale, units = ref.quant_rows(f64(x[good]))
    within(f64(s[good]), scale, scale * 2.0 ** -24, "scale")
    within(f64(q[good]), units, 0.5 + 127 * 2 * 2.0 ** -24, "codes")
