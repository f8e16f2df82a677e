"""The 8-bit operators on the GPU against their 64-bit forms.

Tolerances.  A bf16 result is the nearest to an fp32 value: half a step is 2^-8 of it.
NORM_SHARE: the norm's fp32 value differs from the exact one by the sum's roundings (up to
32 in a lane's chain of squares, 6 + 3 in the joins: 41 * 2^-24, halved by the root), and the
roundings of v, the mean, eps, the root, the quotient and two products (7 * 2^-24): less than
32 * 2^-24.  A code then lies within 1/2 + 127 * 4 * NORM_SHARE of the exact value in units of
its scale (its own error, the row maximum's, and the two of 127 / max and the product).
Products: the integer sum is exact; int -> fp32 and two products make 3 * 2^-24.
"""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_amd as bq
from gpu_cases import DEV, announce, assert_routing_matches, require_gpu
from oracle import group
from oracle import i8_oracle as ref

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
NORM_SHARE = 32 * 2.0 ** -24
PROD_SHARE = 4 * 2.0 ** -24
EPS = 1e-6


def sync():
    torch.cuda.synchronize()


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    err = np.abs(got - want)
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), f"{what} at {worst}: {got[worst]} for {want[worst]}, bound {np.broadcast_to(bound, err.shape)[worst]}"


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


# ---- norm, quantisation and the way back ----

def norm_inputs(T, H, seed):
    g = np.random.default_rng(seed)
    x, r = dev(g.normal(size=(T, H)), torch.bfloat16), dev(3 * g.normal(size=(T, H)), torch.bfloat16)
    return x, r, dev(1 + 0.3 * g.normal(size=H), torch.bfloat16)


def check_norm(x, r, w, s, y, q, qs):
    v, n = ref.norm(f64(x), None if r is None else f64(r), f64(w), EPS)
    if s is not None:
        within(f64(s), v, np.abs(v) * (HALF + 2.0 ** -23), "sum")
    if y is not None:
        within(f64(y), n, np.abs(n) * (HALF + 2 * NORM_SHARE), "y")
    if q is not None:
        _, scale, units = ref.quant_rows(n)
        within(f64(qs), scale, scale * 2 * NORM_SHARE, "scale")
        within(f64(q), units, 0.5 + 127 * 4 * NORM_SHARE, "codes")
        assert int(q.max()) <= 127 and int(q.min()) >= -127


# widths on both sides of every change of waves and pieces per row
@pytest.mark.parametrize("T,H", [(1, 64), (3, 512), (5, 576), (4, 1024), (7, 1088), (1, 2048), (33, 2048),
                                 (2, 2112), (5, 4096), (3, 4160), (2, 7168), (3, 8192), (2, 8256), (1, 16384)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_norm(T, H, with_residual):
    require_gpu()
    announce(f"norm T={T} H={H}")
    x, r, w = norm_inputs(T, H, T * H)
    r = r if with_residual else None
    bf = lambda: torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    s, y = bf(), bf()
    q, qs = torch.zeros((T, H), dtype=torch.int8, device=DEV), torch.zeros(T, device=DEV)
    bq.moe_norm_i8(x, r, w, EPS, s, y, q, qs)
    sync()
    check_norm(x, r, w, s, y, q, qs)
    # each output alone is the same, and the sum may replace an input
    y2, q2, qs2 = bf(), torch.empty_like(q), torch.empty_like(qs)
    bq.moe_norm_i8(x, r, w, EPS, y=y2)
    bq.moe_norm_i8(x, r, w, EPS, q=q2, q_scale=qs2)
    into = x.clone() if r is None else r.clone()
    bq.moe_norm_i8(into if r is None else x, None if r is None else into, w, EPS, into)
    sync()
    assert torch.equal(y, y2) and torch.equal(q, q2) and torch.equal(qs, qs2) and torch.equal(s, into)


def test_norm_of_zeros_and_of_extreme_rows():
    require_gpu()
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device=DEV)
    x[1], x[2] = 1e-20, 1e18
    x[3, 5] = -2.0
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    y, q, qs = torch.empty_like(x), torch.empty((4, 128), dtype=torch.int8, device=DEV), torch.empty(4, device=DEV)
    bq.moe_norm_i8(x, None, w, EPS, None, y, q, qs)
    sync()
    assert not y[0].any() and not q[0].any() and float(qs[0]) == 0
    check_norm(x[1:], None, w, None, y[1:], q[1:], qs[1:])


@pytest.mark.parametrize("R,K", [(1, 64), (6, 512), (9, 1024), (257, 2048), (2, 4096), (3, 8256), (1, 16384)])
def test_quant_and_back(R, K):
    require_gpu()
    announce(f"quant R={R} K={K}")
    x = dev(np.random.default_rng(K).normal(size=(R, K)), torch.bfloat16)
    x[R // 2] = 0
    q, s = torch.zeros((R, K), dtype=torch.int8, device=DEV), torch.full((R,), -1.0, device=DEV)
    out = torch.empty_like(x)
    bq.moe_quant_i8(x, q, s)
    bq.moe_dequant_i8_bf16(q, s, out)
    sync()
    _, scale, units = ref.quant_rows(f64(x))
    within(f64(s), scale, scale * 2.0 ** -24, "scale")            # one division
    within(f64(q), units, 0.5 + 127 * 2 * 2.0 ** -24, "codes")    # a division and a product
    v = f64(q) * f64(s)[:, None]
    within(f64(out), v, np.abs(v) * (HALF + 2.0 ** -23), "values")


def test_rows_on_both_sides_of_the_smallest_scale():
    """127 / max|row| must stay in fp32's range: rows below 2^-119 count as zeros."""
    require_gpu()
    x = torch.zeros((5, 64), dtype=torch.bfloat16, device=DEV)
    for i, v in enumerate((2.0 ** -119, 2.0 ** -120, 2.0 ** -133, 2.0 ** 127, 3e38)):
        x[i, 3], x[i, 9] = v, -v / 2
    q, s = torch.full((5, 64), 5, dtype=torch.int8, device=DEV), torch.empty(5, device=DEV)
    bq.moe_quant_i8(x, q, s)
    sync()
    assert not q[1:3].any() and not s[1:3].any()
    for i in (0, 3, 4):
        assert int(q[i, 3]) == 127 and int(q[i, 9]) in (-63, -64) and int(q[i].abs().sum()) <= 191
        assert float(s[i]) == pytest.approx(float(x[i, 3]) / 127, rel=2.0 ** -22)


def test_dequant_takes_every_code():
    require_gpu()
    q = torch.arange(-128, 128, dtype=torch.int16, device=DEV).to(torch.int8).repeat(5, 1)
    s = torch.tensor([1.0, 0.5, 0.0, -2.0, 1e-30], device=DEV)
    out = torch.empty((5, 256), dtype=torch.bfloat16, device=DEV)
    bq.moe_dequant_i8_bf16(q, s, out)
    sync()
    want = (q.float() * s[:, None]).bfloat16()
    assert torch.equal(out, want)


@pytest.mark.parametrize("R,K", [(1, 64), (3, 1024), (7, 1088), (2047, 2112), (2048, 1088), (2050, 2048), (2500, 64)])
def test_dequant_in_parts_and_by_rows(R, K):
    require_gpu()
    g = np.random.default_rng(R + K)
    q, s = dev(codes(g, R, K), torch.int8), dev(g.normal(size=R), torch.float32)
    out = torch.full((R + 1, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    bq.moe_dequant_i8_bf16(q, s, out[:R])
    sync()
    assert torch.equal(out[:R], (q.float() * s[:, None]).bfloat16()) and out[R].isnan().all()


# ---- scored routing ----

def scored(lg, bias, k, br=32, **rule):
    T, E = lg.shape
    r = bq.DeviceRouting(T, E, k, br, DEV)
    ws = torch.empty(max(bq.route_workspace_bytes(T, E, k, br), 256), dtype=torch.uint8, device=DEV)
    bq.moe_route_scored(dev(lg, torch.float32), None if bias is None else dev(bias, torch.float32),
                        bq.ScoreRule(**rule), k, br, r, ws)
    sync()
    return r.to_host()


def check_scored(lg, bias, k, br=32, score="softmax", **rule):
    announce(f"scored routing {lg.shape} k={k} {score} {rule}")
    got = scored(lg, bias, k, br, score=score, **rule)
    named = dict(rule, top2=rule.get("group_score", "top2") == "top2")
    named.pop("group_score", None)
    named.setdefault("topk_groups", named.get("n_groups", 1))
    idx, w = ref.route_scored(lg, bias, k, sigmoid=score == "sigmoid", **named)
    assert np.array_equal(got["topk_idx"], idx)
    # a score is one rounding; the sum of k, the quotient and the factor are k + 2 more
    within(got["topk_w"].astype(np.float64), w, np.abs(w) * (2 * k + 4) * 2.0 ** -24 + 1e-37, "weights")
    g = group(idx, lg.shape[1], br)
    for key in ("counts", "offsets", "sorted_assign", "assign_row", "block_expert", "block_row"):
        assert np.array_equal(got[key], g[key]), key
    assert int(got["n_blocks"][0]) == int(g["n_blocks"])


# sizes of one launch (T <= 8), of counts from the indices and, above 32768 assignments, of
# segments of 8 (T <= 4096) and 16 tokens; group
# sizes that are whole lanes (32 of 256), that are not (5 of 60, 20 of 160) and groups of one
@pytest.mark.parametrize("T,E,k,n_groups,topk_groups", [
    (1, 256, 8, 8, 4), (1, 1, 1, 1, 1), (5, 2, 2, 1, 1), (64, 64, 6, 8, 3), (65, 256, 8, 8, 4), (33, 60, 5, 12, 4),
    (130, 160, 6, 8, 3), (97, 160, 4, 8, 7), (70, 128, 16, 2, 1), (9, 1000, 10, 10, 3), (66, 1000, 8, 8, 2),
    (2731, 36, 6, 4, 2), (2101, 1000, 8, 8, 2), (1025, 40, 16, 1, 1), (129, 8, 8, 1, 1), (4099, 12, 4, 3, 2),
    (4096, 256, 8, 8, 4), (4097, 256, 8, 8, 4), (8201, 60, 4, 1, 1), (3000, 1000, 16, 8, 2), (4200, 20, 8, 4, 3),
    (2050, 130, 17, 1, 1), (600, 64, 64, 64, 64), (8, 256, 8, 8, 4), (9, 256, 8, 8, 4), (1024, 33, 1, 1, 1), (513, 7, 2, 7, 5),
    (40, 96, 2, 48, 5), (20, 512, 64, 16, 2), (70, 64, 64, 64, 64), (18, 256, 3, 64, 9), (12, 320, 4, 64, 1)])
@pytest.mark.parametrize("score,group_score", [("sigmoid", "top2"), ("softmax", "max"), ("softmax", "top2")])
def test_scored_routing(T, E, k, n_groups, topk_groups, score, group_score):
    require_gpu()
    if group_score == "top2" and E // n_groups < 2:
        group_score = "max"
    g = np.random.default_rng(T * E + k)
    lg = g.normal(size=(T, E)).astype(np.float32)
    bias = (0.1 * g.normal(size=E)).astype(np.float32) if T % 2 else None
    check_scored(lg, bias, k, 16 if T % 3 else 64, score, n_groups=n_groups, topk_groups=topk_groups,
                 group_score=group_score, renormalise=bool(T % 4), scale=2.5 if T % 5 else 1.0)


@pytest.mark.parametrize("T,E,k", [(3000, 40, 8), (5000, 1000, 8)])
def test_scored_routing_of_tokens_that_choose_alike(T, E, k):
    require_gpu()
    lg = np.tile(np.random.default_rng(E).normal(size=E).astype(np.float32), (T, 1))
    check_scored(lg, None, k, 64, "softmax")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [6, 96])
def test_scored_routing_of_masked_and_tied_rows(score, T):
    """Rows of -inf alone, masked experts, NaN, +inf, ties everywhere, scores that vanish in fp32,
    and biases of -inf: the order is the lowest index's, the weights are finite."""
    require_gpu()
    E, inf, nan = 24, np.inf, np.nan
    lg = np.zeros((T, E), np.float32)
    lg[0] = -inf
    lg[1, ::2] = -inf
    lg[2, 3], lg[2, 7], lg[2, 9] = inf, inf, nan
    lg[3] = np.repeat(np.arange(6), 4)
    lg[4] = -200.0
    lg[4, 20] = 5.0
    lg[5] = nan
    bias = np.zeros(E, np.float32)
    check_scored(lg, None, 4, score=score, n_groups=6, topk_groups=3, group_score="top2")
    check_scored(lg, bias, 8, score=score, n_groups=3, topk_groups=2, group_score="max", renormalise=False)
    bias[[0, 1, 2, 3, 11]] = -inf
    check_scored(lg, bias, 5, score=score)
    check_scored(lg, bias, 4, score=score, n_groups=6, topk_groups=2, group_score="top2")
    check_scored(lg, np.full(E, -inf, np.float32), 4, score=score, n_groups=6, topk_groups=6)


def test_softmax_rule_without_bias_selects_as_moe_route():
    require_gpu()
    lg = np.random.default_rng(5).normal(size=(200, 256)).astype(np.float32)
    assert_routing_matches(scored(lg, None, 8), lg, 8)


# ---- products ----

def codes(g, *shape):
    return g.integers(-127, 128, shape).astype(np.int8)


def i8mat(q, s, layout):
    m = bq.DeviceI8Mat(dev(q, torch.int8), dev(s, torch.float32))
    return m.prepacked() if layout else m


def test_prepack_order():
    require_gpu()
    q = codes(np.random.default_rng(0), 3, 48, 192)
    got = i8mat(q, np.ones((3, 48), np.float32), 1).codes.cpu().numpy()
    want = q.reshape(3, 3, 16, 3, 4, 16).transpose(0, 1, 3, 4, 2, 5).reshape(3, 48, 192)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 64), (1, 16, 64), (1, 4096, 2048), (2, 33, 128), (15, 100, 192), (16, 16, 512), (17, 16, 512),
    (33, 65, 320), (64, 128, 256), (65, 129, 64), (100, 250, 448), (128, 256, 128), (129, 272, 576),
    # K split over the waves of a workgroup: 16 x 32, 32 x 32 and 32 x 64
    (33, 1411, 320), (50, 1440, 192), (20, 4096, 64), (45, 4064, 192), (64, 4096, 64), (64, 4080, 1088), (100, 4000, 576),
    (128, 4096, 2048), (97, 4048, 64), (250, 2000, 1088),
    # each tile of the many-row kernel, with ragged edges, N in and out of eights, K of one block,
    # of an odd number and of many; the last three take several tiles a workgroup
    (300, 1500, 192), (333, 1001, 64), (700, 1000, 320), (650, 999, 1088), (1100, 1411, 320),
    (1030, 1480, 64), (1500, 1411, 320), (1536, 1408, 576), (3500, 3841, 192), (3585, 3600, 64),
    (2000, 4000, 1088), (2200, 4090, 320), (8000, 4360, 64), (4400, 4360, 128), (4400, 4365, 64), (70000, 100, 64), (255, 1001, 192), (256, 256, 1024), (300, 528, 704), (513, 768, 320), (1, 100, 8192), (40, 48, 16384)])
@pytest.mark.parametrize("layout", [0, 1])
def test_linear(M, N, K, layout):
    require_gpu()
    if layout and N % 16:
        N = (N + 15) // 16 * 16
    announce(f"linear M={M} N={N} K={K} layout={layout}")
    g = np.random.default_rng(M * N + K)
    a, w = codes(g, M, K), codes(g, 1, N, K)
    sa, sw = g.random(M).astype(np.float32), g.random((1, N)).astype(np.float32)
    # rows behind the last and bytes behind the output stay as they were
    out = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(256, bq.linear_i8_workspace_bytes(M, N, K)), dtype=torch.uint8, device=DEV)
    bq.moe_linear_i8(dev(a, torch.int8), dev(sa, torch.float32), i8mat(w, sw, layout), out[:M * N].view(M, N), ws)
    sync()
    want = ref.linear(a, sa, w[0], sw[0])
    within(f64(out[:M * N]).reshape(M, N), want, np.abs(want) * (HALF + PROD_SHARE), "out")
    assert (out[M * N:] == 7.0).all()


def test_linear_of_extreme_codes_is_exact():
    """-128 on both sides over the longest K: the sum, 128 * 128 * 131008, still fits 32 bits."""
    require_gpu()
    K = 131072 - 64
    for M in (1, 80):
        a = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
        w = bq.DeviceI8Mat(torch.full((1, 32, K), -128, dtype=torch.int8, device=DEV), torch.ones((1, 32), device=DEV))
        out = torch.empty((M, 32), dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(max(256, bq.linear_i8_workspace_bytes(M, 32, K)), dtype=torch.uint8, device=DEV)
        bq.moe_linear_i8(a, torch.ones(M, device=DEV), w, out, ws)
        sync()
        assert (out.double() == torch.tensor(float(16384 * K)).bfloat16().double().item()).all()


# ---- the experts' products, the layer, the block ----

def layer_weights(g, E, H, I, I_sh):
    shapes = [(E, I, H), (E, I, H), (E, H, I)] + ([(1, I_sh, H), (1, I_sh, H), (1, H, I_sh)] if I_sh else [])
    # scales that keep |x Wg^T| below 32: 127 codes of at most 1/127 * sqrt(3 / K) * 4
    return [(codes(g, *s), (g.uniform(0.3, 1.0, s[:2]) / 127 * (3.0 / s[2]) ** 0.5).astype(np.float32))
            for s in shapes]


def check_layer(got, x, sx, idx, w, host, I_sh, what):
    k, H = idx.shape[1], x.shape[1]
    T = x.shape[0]
    eo, b, sh, b_sh, y = ref.layer(x, sx, idx, w, host[:3], host[3:] if I_sh else None)
    rows = got["routing"].assign_row.cpu().numpy()
    b = b + np.abs(eo) * PROD_SHARE
    bound = HALF * (np.abs(eo) + b) + b
    if "expert_out" in got["checked"]:
        within(f64(got["expert_out"])[rows], eo, bound, what + " expert_out")
    total = (bound.reshape(T, k, H) * w[:, :, None]).sum(1)
    size = (np.abs(eo).reshape(T, k, H) * w[:, :, None]).sum(1)
    if I_sh:
        b_sh = HALF * (np.abs(sh) + b_sh) + b_sh + np.abs(sh) * PROD_SHARE
        if "shared_out" in got["checked"]:
            within(f64(got["shared_out"]), sh, b_sh, what + " shared_out")
        total, size = total + b_sh, size + np.abs(sh)
    # fp32 weights (1e-6 as for moe_route), the fp32 sum, one rounding to bf16
    total = total + size * (1e-6 + (k + 2) * 2.0 ** -23)
    within(f64(got["y"]), y, total + HALF * (np.abs(y) + total), what + " y")


LAYERS = [  # T, H, I, I_sh, E, k
    (1, 64, 64, 0, 4, 1), (1, 256, 128, 128, 16, 4), (1, 2048, 512, 512, 16, 8), (1, 128, 1088, 64, 70, 20), (1, 192, 4160, 0, 4, 2), (1, 64, 4096, 64, 32, 17), (3, 256, 128, 64, 60, 4), (8, 2048, 512, 512, 256, 8), (2, 192, 64, 320, 8, 3), (7, 256, 192, 64, 16, 2),
    (33, 320, 128, 0, 6, 6), (65, 512, 64, 128, 60, 4), (130, 128, 448, 64, 16, 8), (257, 256, 128, 192, 4, 2),
    (40, 64, 1088, 1152, 3, 2), (9, 64, 640, 64, 6, 2), (5, 128, 2112, 576, 6, 2),
    (64, 128, 64, 64, 16, 2), (40, 1024, 256, 0, 16, 2), (24, 2048, 512, 512, 16, 8)]


@pytest.mark.parametrize("T,H,I,I_sh,E,k", LAYERS)
@pytest.mark.parametrize("block_rows,layout", [(16, 1), (32, 0), (32, 1), (64, 1)])
def test_layer(T, H, I, I_sh, E, k, block_rows, layout):
    require_gpu()
    what = f"layer T={T} H={H} I={I} I_sh={I_sh} E={E} k={k} rows={block_rows} layout={layout}"
    announce(what)
    g = np.random.default_rng(T + H + I)
    host = layer_weights(g, E, H, I, I_sh)
    x, sx = codes(g, T, H), g.uniform(0.01, 0.03, T).astype(np.float32)
    lg = g.normal(size=(T, E)).astype(np.float32)
    lg[:, 0] += 1.5   # unequal experts: some with several blocks, some empty
    mats = [i8mat(q, s, layout) for q, s in host] + [None] * (6 - len(host))
    layer = bq.MoeLayerI8(mats, H, I, I_sh, E, k, DEV, block_rows=block_rows)
    b = layer.buffers(T)
    for name in ("expert_out", "shared_out", "y"):
        if b[name] is not None:
            b[name].fill_(float("nan"))
    xd, sd, ld = dev(x, torch.int8), dev(sx, torch.float32), dev(lg, torch.float32)
    few = T <= 64   # may leave expert_out and shared_out alone
    got = dict(layer.forward(xd, sd, ld), checked=() if few else ("expert_out", "shared_out"))
    sync()
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :k].astype(np.int32)
    p = np.exp(np.take_along_axis(lg, idx, 1).astype(np.float64))
    w = p / p.sum(1, keepdims=True)
    check_layer(got, x, sx, idx, w, host, I_sh, what)
    assert_routing_matches(got["routing"].to_host(), lg, k, block_rows)
    # the three calls on their own give the layer call's result
    y = got["y"].clone()
    r = got["routing"]
    bq.moe_grouped_gemm_i8(xd, sd, I, I_sh, E, k, block_rows, r, *mats, b["expert_out"], b["shared_out"], b["gemm_ws"])
    y3 = torch.empty_like(y)
    bq.moe_combine(b["expert_out"], b["shared_out"], r, k, y3)
    sync()
    check_layer(dict(got, y=y3, checked=("expert_out", "shared_out")), x, sx, idx, w, host, I_sh, what + ", three calls")
    # the same call again, and into another output: bit for bit
    again = torch.empty_like(y)
    layer.forward(xd, sd, ld, out=again)
    sync()
    assert torch.equal(again, y)


@pytest.mark.parametrize("T", [1, 3, 70])
def test_block_runs_norm_router_scored_routing_and_layer(T):
    """The operators in a run, as a model's block has them: each stage against its 64-bit form over
    the stage before's own output."""
    require_gpu()
    announce(f"block T={T}")
    H, I, I_sh, E, k = 256, 128, 64, 32, 4
    g = np.random.default_rng(T)
    host = layer_weights(g, E, H, I, I_sh)
    bias = (0.05 * g.normal(size=E)).astype(np.float32)
    rule = dict(score="sigmoid", n_groups=4, topk_groups=2, scale=1.5)
    layer = bq.MoeLayerI8([i8mat(q, s, 1) for q, s in host], H, I, I_sh, E, k, DEV,
                          rule=bq.ScoreRule(**rule), score_bias=dev(bias, torch.float32))
    x, r, w = norm_inputs(T, H, 3)
    router = dev(g.normal(size=(E, H)) * H ** -0.5, torch.bfloat16)
    got = layer.forward_block(x, r, w, router)
    sync()
    check_norm(x, r, w, got["sum"], got["normed"], got["q"], got["q_scale"])
    lg = got["logits"].cpu().numpy()
    want = f64(got["normed"]) @ f64(router).T
    # fp32 sums of H products of bf16 values
    within(lg.astype(np.float64), want, H * 2.0 ** -23 * (np.abs(f64(got["normed"])) @ np.abs(f64(router)).T), "logits")
    idx, wgt = ref.route_scored(lg, bias, k, sigmoid=True, n_groups=4, topk_groups=2, scale=1.5)
    assert np.array_equal(got["routing"].topk_idx.cpu().numpy(), idx)
    check_layer(dict(got, checked=()), got["q"].cpu().numpy(), got["q_scale"].cpu().numpy(), idx, wgt, host, I_sh, "block")


def test_from_bf16_quantises_by_channel():
    require_gpu()
    H, I, E, k = 128, 64, 4, 2
    g = np.random.default_rng(9)
    w = [dev(g.normal(size=s), torch.bfloat16) for s in ((E, I, H), (E, I, H), (E, H, I))]
    layer = bq.MoeLayerI8.from_bf16(w + [None] * 3, H, I, 0, E, k, DEV)
    sync()
    for m, v in zip(layer.mats[:3], w):
        n, N, K = v.shape
        _, scale, units = ref.quant_rows(f64(v))
        got = m.codes.view(n, N // 16, K // 64, 4, 16, 16).permute(0, 1, 4, 2, 3, 5).reshape(n, N, K)
        within(f64(got), units, 0.5 + 127 * 2 * 2.0 ** -24, "codes")
        within(f64(m.scales), scale, scale * 2.0 ** -24, "scales")


@pytest.mark.parametrize("T", [1, 80])
def test_captured_block_replays_as_the_eager_one(T):
    """A graph of the whole block over new inputs, between eager calls of another layer object."""
    require_gpu()
    announce(f"captured block T={T}")
    H, I, I_sh, E, k = 256, 128, 64, 32, 4
    g = np.random.default_rng(1)
    host = layer_weights(g, E, H, I, I_sh)
    mats = [i8mat(q, s, 1) for q, s in host]
    captured, eager = (bq.MoeLayerI8(mats, H, I, I_sh, E, k, DEV, rule=bq.ScoreRule("sigmoid")) for _ in range(2))
    router = dev(g.normal(size=(E, H)) * H ** -0.5, torch.bfloat16)
    x, r, w = norm_inputs(T, H, 0)
    captured.forward_block(x, r, w, router)   # its buffers, before the capture
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured.forward_block(x, r, w, router)
    for seed in range(4):
        nx, nr, _ = norm_inputs(T, H, 10 + seed)
        x.copy_(nx)
        r.copy_(nr)
        graph.replay()
        want = eager.forward_block(nx, nr, w, router)
        sync()
        for name in ("sum", "normed", "q", "q_scale", "logits", "y"):
            assert torch.equal(out[name], want[name]), (seed, name)


def test_two_streams_with_an_object_each():
    require_gpu()
    H, I, I_sh, E, k, T = 256, 128, 64, 16, 2, 50
    g = np.random.default_rng(2)
    host = layer_weights(g, E, H, I, I_sh)
    mats = [i8mat(q, s, 1) for q, s in host]
    xs = [(dev(codes(g, T, H), torch.int8), dev(g.random(T), torch.float32) * 0.02,
           dev(g.normal(size=(T, E)), torch.float32)) for _ in range(2)]
    layers = [bq.MoeLayerI8(mats, H, I, I_sh, E, k, DEV) for _ in range(2)]
    want = [layer.forward(*x)["y"].clone() for layer, x in zip(layers, xs)]
    sync()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for layer, x, st in zip(layers, xs, streams):
            layer.forward(*x, stream=st)
    sync()
    for layer, v in zip(layers, want):
        assert torch.equal(layer.buffers(T)["y"], v)


def test_new_buffers_wait_for_the_current_stream():
    """A first call on another stream allocates from the current stream's memory: it must not run
    before what is enqueued there."""
    require_gpu()
    H, I, E, k, T = 256, 128, 16, 2, 50
    g = np.random.default_rng(5)
    host = layer_weights(g, E, H, I, 0)
    mats = [i8mat(q, s, 1) for q, s in host] + [None] * 3
    x, r, w = norm_inputs(T, H, 4)
    router = dev(g.normal(size=(E, H)) * H ** -0.5, torch.bfloat16)
    bf = dev(g.normal(size=(E, I, H)), torch.bfloat16)
    want = bq.MoeLayerI8(mats, H, I, 0, E, k, DEV).forward_block(x, r, w, router)
    want_mat = bq.DeviceI8Mat.from_bf16(bf)
    big = torch.zeros(1 << 28, device=DEV)
    side = torch.cuda.Stream()
    sync()

    def behind_work(call):
        done = torch.cuda.Event()
        for _ in range(20):
            big.add_(1.0)   # 2 GiB of traffic each, about 8 ms in all
        done.record()
        out = call()
        side.synchronize()
        assert done.query()
        return out

    layer = bq.MoeLayerI8(mats, H, I, 0, E, k, DEV)
    got = behind_work(lambda: layer.forward_block(x, r, w, router, stream=side))
    other = bq.MoeLayerI8(mats, H, I, 0, E, k, DEV)
    y = behind_work(lambda: other.forward(want["q"], want["q_scale"], want["logits"], stream=side))["y"]
    m = behind_work(lambda: bq.DeviceI8Mat.from_bf16(bf, stream=side))
    sync()
    assert torch.equal(got["y"], want["y"]) and torch.equal(y, want["y"])
    assert torch.equal(m.codes, want_mat.codes) and torch.equal(m.scales, want_mat.scales)


@pytest.mark.parametrize("T", [1, 3, 100])
def test_matrices_of_both_layouts_in_one_call(T):
    """Only gate and up (and the shared two) need the same layout; every mix gives the same bits."""
    require_gpu()
    H, I, I_sh, E, k = 256, 128, 192, 64, 4
    g = np.random.default_rng(T)
    host = layer_weights(g, E, H, I, I_sh)
    x, sx = dev(codes(g, T, H), torch.int8), dev(g.random(T), torch.float32) * 0.02
    lg = dev(g.normal(size=(T, E)), torch.float32)
    ys = []
    for pair, down, sh_pair, sh_down in ((1, 1, 1, 1), (1, 0, 0, 1), (0, 1, 1, 0)):
        mats = [i8mat(q, s, v) for (q, s), v in zip(host, (pair, pair, down, sh_pair, sh_pair, sh_down))]
        ys.append(bq.MoeLayerI8(mats, H, I, I_sh, E, k, DEV).forward(x, sx, lg)["y"].clone())
    sync()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


@pytest.mark.parametrize("M", [3, 200])
def test_scales_need_four_bytes_alignment_only(M):
    require_gpu()
    N, K, E = 64, 128, 3
    g = np.random.default_rng(M)
    wq, ws = dev(codes(g, E, N, K), torch.int8), dev(g.random((E, N)) * 0.01, torch.float32)
    odd = torch.empty(E * N + 1, device=DEV)[1:].view(E, N)
    odd.copy_(ws)
    x, sx = dev(codes(g, M, K), torch.int8), dev(g.random(M), torch.float32)
    odd_sx = torch.empty(M + 1, device=DEV)[1:]
    odd_sx.copy_(sx)
    outs = [torch.empty((M, N), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    bq.moe_linear_i8(x, sx, bq.DeviceI8Mat(wq[:1], ws[:1]), outs[0])
    bq.moe_linear_i8(x, odd_sx, bq.DeviceI8Mat(wq[:1], odd[:1]), outs[1])
    down = dev(codes(g, E, K, N), torch.int8), dev(g.random((E, K)) * 0.01, torch.float32)
    lg, ys = dev(g.normal(size=(M, E)), torch.float32), []
    for s, rs in ((ws, sx), (odd, odd_sx)):
        m = bq.DeviceI8Mat(wq, s)
        layer = bq.MoeLayerI8([m, m, bq.DeviceI8Mat(*down)] + [None] * 3, K, N, 0, E, 2, DEV)
        ys.append(layer.forward(x, rs, lg)["y"])
    sync()
    assert torch.equal(*outs) and torch.equal(*ys)


# ---- sizes at which offsets pass 31 and 32 bits, and variants chosen by size ----

@pytest.mark.parametrize("with_residual", [True, False])
def test_streamed_norm_equals_the_cached_one(with_residual):
    """Inputs over 128 MB take non-temporal loads; slices of the same rows do not."""
    require_gpu()
    T, H = (8200, 4160) if with_residual else (16400, 4160)
    announce(f"norm T={T} H={H}")
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((T, H), device=DEV, generator=g).bfloat16()
    r = torch.randn((T, H), device=DEV, generator=g).bfloat16() if with_residual else None
    w = torch.randn(H, device=DEV, generator=g).bfloat16()
    out = lambda n: (torch.empty((n, H), dtype=torch.bfloat16, device=DEV), torch.empty((n, H), dtype=torch.bfloat16, device=DEV),  # noqa: E731
                     torch.empty((n, H), dtype=torch.int8, device=DEV), torch.empty(n, device=DEV))
    whole, q, qs = out(T), torch.empty((T, H), dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    bq.moe_norm_i8(x, r, w, EPS, *whole)
    bq.moe_quant_i8(x, q, qs)
    for at in (0, T // 2, T - 77):
        part, pq, ps = out(77), torch.empty((77, H), dtype=torch.int8, device=DEV), torch.empty(77, device=DEV)
        bq.moe_norm_i8(x[at:at + 77], None if r is None else r[at:at + 77], w, EPS, *part)
        bq.moe_quant_i8(x[at:at + 77], pq, ps)
        sync()
        for a, b in zip(whole + (q, qs), part + (pq, ps)):
            assert torch.equal(a[at:at + 77], b)


def test_rows_past_32_bit_offsets():
    require_gpu()
    R, K = 131073 + 5, 16384   # 2^31 elements and some
    announce(f"quant R={R} K={K}")
    x = torch.zeros((R, K), dtype=torch.bfloat16, device=DEV)
    x[-1] = torch.arange(K, device=DEV).remainder(255).sub(127).bfloat16()
    q, s = torch.full((R, K), 1, dtype=torch.int8, device=DEV), torch.full((R,), -1.0, device=DEV)
    out = torch.full((R, K), 1.0, dtype=torch.bfloat16, device=DEV)
    bq.moe_quant_i8(x, q, s)
    bq.moe_dequant_i8_bf16(q, s, out)
    sync()
    assert float(s[-1]) == 1.0 and torch.equal(q[-1].float(), x[-1].float()) and torch.equal(out[-1], x[-1])
    assert not q[-2].any() and float(s[0]) == 0 and not out[R // 2].any()


def test_dequant_of_the_widest_row():
    require_gpu()
    K = (1 << 31) - 64
    q = torch.full((1, K), 3, dtype=torch.int8, device=DEV)
    q[0, -1] = -7
    out = torch.zeros((1, K), dtype=torch.bfloat16, device=DEV)
    bq.moe_dequant_i8_bf16(q, torch.full((1,), 0.5, device=DEV), out)
    sync()
    assert float(out[0, -1]) == -3.5 and bool((out[0, :-1] == 1.5).all())


def test_linear_of_outputs_past_31_bits():
    require_gpu()
    M, N, K = 33_500_000, 66, 64   # M * N = 2.2e9
    announce(f"linear M={M} N={N} K={K}")
    a = torch.zeros((M, K), dtype=torch.int8, device=DEV)
    a[-1] = 1
    w = bq.DeviceI8Mat(torch.arange(N, device=DEV, dtype=torch.int8).view(1, N, 1).expand(1, N, K).contiguous(),
                       torch.ones((1, N), device=DEV))
    out = torch.full((M, N), 9.0, dtype=torch.bfloat16, device=DEV)
    bq.moe_linear_i8(a, torch.ones(M, device=DEV), w, out)
    sync()
    assert torch.equal(out[-1].float(), 64 * torch.arange(N, device=DEV).float())
    assert not out[0].any() and not out[M // 2].any() and not out[-2].any()


def test_large_layer_equals_its_slices():
    """A token's sums do not depend on the others, and the integer sums are exact: the same tokens
    in a call of 40000 (2^31 bytes of expert rows and more) and in calls of any block size."""
    require_gpu()
    T, H, I, I_sh, E, k = 40000, 2048, 256, 128, 64, 8
    announce(f"layer T={T}")
    g = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda *s: torch.randint(-127, 128, s, device=DEV, generator=g, dtype=torch.int8)  # noqa: E731
    mats = [bq.DeviceI8Mat(rnd(*s), torch.rand(s[:2], device=DEV, generator=g) * 1e-3)
            for s in ((E, I, H), (E, I, H), (E, H, I), (1, I_sh, H), (1, I_sh, H), (1, H, I_sh))]
    x, sx = rnd(T, H), torch.rand(T, device=DEV, generator=g) * 0.02
    lg = torch.randn((T, E), device=DEV, generator=g)
    whole = bq.MoeLayerI8(mats, H, I, I_sh, E, k, DEV).forward(x, sx, lg)["y"]
    for at, n, rows in ((0, 40, 16), (20000, 300, 32), (39000, 1000, 32), (37000, 3000, 64)):
        part = bq.MoeLayerI8(mats, H, I, I_sh, E, k, DEV, block_rows=rows)
        y = part.forward(x[at:at + n], sx[at:at + n], lg[at:at + n])["y"]
        sync()
        assert torch.equal(whole[at:at + n], y), (at, n, rows)
