"""moe_decode_batch_q4's selection inside the first launch (1 to 8 tokens) at every number of experts a
lane holds, and on both sides of the changes of its method."""
import pytest

import bit_quantized_grouped_amd as bq
import test_gpu_batch as tb
from gpu_cases import require_gpu

pytestmark = pytest.mark.gpu

# experts of 1, 2, 4, 8 and 16 a lane, and both ends of each
EXPERTS = [63, 64, 65, 128, 129, 130, 160, 256, 257, 512, 513, 600, 1000]


@pytest.mark.parametrize("T", [1, 2, 5, 8])
@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("layout", [bq.LAYOUT_ROWS, bq.LAYOUT_TILES_SB])
def test_every_number_of_experts_a_lane(T, E, layout):
    require_gpu()
    tb.check_call(T, 128, 64, 64, E, 6, layout, gated=True)


# 16 is the last k of rounds, 17 the first of the radix selection, whose scratch lies behind the masks
@pytest.mark.parametrize("T", [1, 5, 8])
@pytest.mark.parametrize("E,k", [(60, 17), (100, 64), (130, 17), (256, 16), (256, 33), (256, 64), (500, 64), (600, 17), (1000, 16),
                                 (1000, 64)])
@pytest.mark.parametrize("layout", [bq.LAYOUT_ROWS, bq.LAYOUT_TILES_SB])
def test_many_experts_a_token(T, E, k, layout):
    require_gpu()
    tb.check_call(T, 64, 64, 0, E, k, layout)


@pytest.mark.parametrize("T", [1, 2, 8])
@pytest.mark.parametrize("E,k,rule", [
    (130, 6, dict(score="sigmoid", n_groups=10, topk_groups=3)), (160, 8, dict(score="softmax", n_groups=8, topk_groups=3, scale=4.0)),
    (256, 8, dict(score="sigmoid", n_groups=8, topk_groups=4, scale=2.5)), (256, 64, dict(score="softmax", renormalise=False)),
    (600, 20, dict(score="sigmoid", n_groups=12, topk_groups=2, group_score="max")), (1000, 64, dict(score="sigmoid")),
    (1000, 9, dict(score="softmax", n_groups=8, topk_groups=1))])
def test_scored_selection_of_many_experts(T, E, k, rule):
    require_gpu()
    tb.check_call(T, 64, 128, 64, E, k, bq.LAYOUT_TILES_SB, rule=rule, gated=True)
