"""The 8-bit operators on the GPU at the edges of what they take.

Tolerances are those of test_gpu_i8.py, whose helpers and 64-bit forms these tests use.
"""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_amd as bq
from gpu_cases import DEV, announce, assert_routing_matches, require_gpu
from oracle import i8_oracle as ref
from test_gpu_i8 import (EPS, HALF, PROD_SHARE, check_norm, codes, dev, f64, i8mat, layer_weights, norm_inputs, sync,
                         within)

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


def nan_layer(T, H, I, I_sh, E, k, block_rows):
    """A layer with NaN in a token's scale, in a channel of one expert's gate and an infinity in a
    channel of another's up: (y with them, y without, the tokens that they reach, both dicts)."""
    g = np.random.default_rng(T + I)
    host = layer_weights(g, E, H, I, I_sh)
    x, lg = dev(codes(g, T, H), torch.int8), dev(g.normal(size=(T, E)), torch.float32)
    sx = dev(g.uniform(0.01, 0.03, T), torch.float32)
    mats = [i8mat(q, s, 1) for q, s in host] + [None] * (6 - len(host))
    clean = bq.MoeLayerI8(mats, H, I, I_sh, E, k, DEV, block_rows=block_rows)
    want = clean.forward(x, sx, lg)
    idx = want["routing"].topk_idx
    t_bad = T // 2
    e_nan, e_inf = int(idx[0, 0]), int(idx[0, -1])
    sx2 = sx.clone()
    sx2[t_bad] = NAN
    gate, up = (bq.DeviceI8Mat(m.codes, m.scales.clone(), m.layout) for m in mats[:2])
    gate.scales[e_nan, I - 1] = NAN
    up.scales[e_inf, 0] = INF
    other = bq.MoeLayerI8([gate, up] + mats[2:], H, I, I_sh, E, k, DEV, block_rows=block_rows)
    got = other.forward(x, sx2, lg)
    sync()
    reached = ((idx == e_nan) | (idx == e_inf)).any(1)
    reached[t_bad] = True
    return got["y"], want["y"], reached, got, want


# h by a wave a row, one to eight pieces a lane, and by a workgroup a row; blocks of every size
@pytest.mark.parametrize("I,I_sh,block_rows", [(64, 0, 16), (448, 192, 32), (1024, 64, 32), (1088, 0, 64), (2112, 576, 16),
                                               (64, 2112, 64)])
def test_nan_reaches_the_grouped_layers_output(I, I_sh, block_rows):
    require_gpu()
    announce(f"grouped layer with NaN I={I} I_sh={I_sh} rows={block_rows}")
    T, k = 70, 2
    y, want, reached, got, clean = nan_layer(T, 128, I, I_sh, 24, k, block_rows)
    assert not reached.all() and y[reached].isnan().all() and torch.equal(y[~reached], want[~reached])
    # a row of an expert or of the shared expert is NaN as a whole or what it is without
    for name in ("expert_out", "shared_out") if I_sh else ("expert_out",):
        rows = got[name].isnan().any(1)
        assert got[name][rows].isnan().all() and torch.equal(got[name][~rows], clean[name][~rows])


# h in registers (512 and less) and read twice; more slots than waves
@pytest.mark.parametrize("T,I,I_sh,E,k", [(1, 64, 0, 8, 2), (1, 512, 1088, 8, 3), (1, 1088, 64, 40, 20), (3, 128, 64, 64, 2),
                                          (12, 576, 0, 64, 4)])
def test_nan_reaches_the_output_of_few_tokens(T, I, I_sh, E, k):
    require_gpu()
    announce(f"layer of few tokens with NaN T={T} I={I} I_sh={I_sh}")
    y, want, reached, _, _ = nan_layer(T, 128, I, I_sh, E, k, None)
    assert y[reached].isnan().all() and torch.equal(y[~reached], want[~reached])


# ---- the sum over the experts ----

@pytest.mark.parametrize("T,H,I,I_sh,E,k,block_rows", [
    (70, 256, 128, 0, 6, 6, 16), (130, 128, 448, 64, 16, 8, 32), (300, 320, 64, 192, 8, 4, 64), (80, 1024, 64, 64, 4, 1, 16),
    (200, 2112, 64, 0, 16, 12, 32), (96, 64, 320, 64, 70, 20, 16), (150, 192, 128, 128, 5, 3, 64)])
def test_layer_sums_its_experts_before_rounding(T, H, I, I_sh, E, k, block_rows):
    """y is one rounding of a sum in fp32, as it is for few tokens: an expert's output enters it
    within 2^-15 of itself, where one rounded to bf16 would be 2^-9 of itself off."""
    require_gpu()
    what = f"layer sum T={T} H={H} I={I} I_sh={I_sh} E={E} k={k} rows={block_rows}"
    announce(what)
    g = np.random.default_rng(T * H + I)
    host = layer_weights(g, E, H, I, I_sh)
    x, sx = codes(g, T, H), g.uniform(0.01, 0.03, T).astype(np.float32)
    lg = g.normal(size=(T, E)).astype(np.float32)
    mats = [i8mat(q, s, 1) for q, s in host] + [None] * (6 - len(host))
    layer = bq.MoeLayerI8(mats, H, I, I_sh, E, k, DEV, block_rows=block_rows)
    got = layer.forward(dev(x, torch.int8), dev(sx, torch.float32), dev(lg, torch.float32))
    sync()
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :k].astype(np.int32)
    p = np.exp(np.take_along_axis(lg, idx, 1).astype(np.float64))
    w = p / p.sum(1, keepdims=True)
    eo, b, sh, b_sh, y = ref.layer(x, sx, idx, w, host[:3], host[3:] if I_sh else None)
    # the expert's own error (codes of h at a border, fp32 products), its 2^-15, the fp32 weight
    # (1e-6 as for moe_route) and the fp32 sum of k + 1
    share = PROD_SHARE + 2.0 ** -15 + 1e-6 + (k + 2) * 2.0 ** -23
    bound = ((b + np.abs(eo) * share).reshape(T, k, H) * w[:, :, None]).sum(1)
    if I_sh:
        bound = bound + b_sh + np.abs(sh) * share
    within(f64(got["y"]), y, bound + HALF * (np.abs(y) + bound), what)
    # the experts' rows of the call are still the grouped product's, in bf16
    r = got["routing"]
    eo2, so2 = torch.empty_like(got["expert_out"]), None if not I_sh else torch.empty_like(got["shared_out"])
    ws = torch.empty(bq.gemm_i8_workspace_bytes(T, H, I, I_sh, E, k, block_rows), dtype=torch.uint8, device=DEV)
    bq.moe_grouped_gemm_i8(dev(x, torch.int8), dev(sx, torch.float32), I, I_sh, E, k, block_rows, r, *mats, eo2, so2, ws)
    sync()
    assert torch.equal(eo2, got["expert_out"]) and (so2 is None or torch.equal(so2, got["shared_out"]))


# ---- sizes beyond one launch (a grid dimension ends below 2^32 threads) ----

@pytest.fixture
def large():
    require_gpu()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


# a wave a row, and four waves a row
@pytest.mark.parametrize("R,K", [((1 << 26) + 5, 64), ((1 << 24) + 5, 1088)])
def test_norm_and_quant_of_rows_beyond_one_launch(large, R, K):
    announce(f"norm and quant R={R} K={K}")
    x = torch.zeros((R, K), dtype=torch.bfloat16, device=DEV)
    some = [0, (1 << 21) - 1, 1 << 21, R // 2, R - 1]
    rows = dev(np.random.default_rng(K).normal(size=(len(some), K)), torch.bfloat16)
    x[some] = rows
    w = dev(1 + 0.3 * np.random.default_rng(1).normal(size=K), torch.bfloat16)
    q, s = torch.full((R, K), 1, dtype=torch.int8, device=DEV), torch.full((R,), -1.0, device=DEV)
    want = [torch.empty((len(some), K), dtype=torch.int8, device=DEV), torch.empty(len(some), device=DEV)]
    for call, few in ((lambda: bq.moe_quant_i8(x, q, s), lambda: bq.moe_quant_i8(rows, *want)),
                      (lambda: bq.moe_norm_i8(x, None, w, EPS, q=q, q_scale=s),
                       lambda: bq.moe_norm_i8(rows, None, w, EPS, q=want[0], q_scale=want[1]))):
        q.fill_(1)
        s.fill_(-1.0)
        call()
        few()
        sync()
        assert torch.equal(q[some], want[0]) and torch.equal(s[some], want[1])
        assert int((s != 0).sum()) == len(some)
        s[some] = 0
        q[some] = 0
        assert not any(part.any() for part in q.split(1 << 22))


def test_dequant_of_rows_beyond_one_launch(large):
    R, K = (1 << 26) + 5, 64
    announce(f"dequant R={R} K={K}")
    q, s = torch.zeros((R, K), dtype=torch.int8, device=DEV), torch.ones(R, device=DEV)
    some = [0, (1 << 21) - 1, 1 << 21, R // 2, R - 1]
    q[some], s[some] = 100, torch.arange(1.0, 6.0, device=DEV)
    out = torch.full((R, K), 3.0, dtype=torch.bfloat16, device=DEV)
    bq.moe_dequant_i8_bf16(q, s, out)
    sync()
    assert torch.equal(out[some].float(), (100.0 * torch.arange(1.0, 6.0, device=DEV))[:, None].expand(5, K).bfloat16().float())
    out[some] = 0
    assert not any(part.any() for part in out.split(1 << 22))


def test_dequant_of_few_rows_beyond_one_launch(large):
    """2^21 parts of a row of 1024 codes: 16 rows a launch."""
    R, K = 17, (1 << 31) - 64
    announce(f"dequant R={R} K={K}")
    q, s = torch.zeros((R, K), dtype=torch.int8, device=DEV), torch.ones(R, device=DEV)
    q[:, 0], q[:, K - 1], q[15, 5], q[16, 1 << 30] = 1, 2, 3, 4
    out = torch.full((R, K), 9.0, dtype=torch.bfloat16, device=DEV)
    bq.moe_dequant_i8_bf16(q, s, out)
    sync()
    assert (out[:, 0] == 1).all() and (out[:, K - 1] == 2).all() and float(out[15, 5]) == 3 and float(out[16, 1 << 30]) == 4
    out[:, 0], out[:, K - 1], out[15, 5], out[16, 1 << 30] = 0, 0, 0, 0
    assert not any(part.any() for row in out for part in row.split(1 << 28))


def test_prepack_beyond_one_launch(large):
    """More than 2^32 pieces of 16 codes."""
    E, N, K = 65, 16384, 65536
    announce(f"prepack {E} x {N} x {K}")
    src = torch.zeros((E, N, K), dtype=torch.int8, device=DEV)
    dst = torch.full((E, N, K), 7, dtype=torch.int8, device=DEV)
    some = (0, 15, 16, 33, 64)   # a launch takes 2^30 pieces, 16 matrices
    for e in some:
        src[e] = torch.randint(-128, 128, (N, K), dtype=torch.int8, device=DEV, generator=torch.Generator(DEV).manual_seed(e))
    bq.moe_i8_prepack(src, dst)
    sync()
    for e in range(E):
        if e in some:
            want = src[e].view(N // 16, 16, K // 64, 4, 16).permute(0, 2, 3, 1, 4).reshape(N, K)
            assert torch.equal(dst[e], want), e
        else:
            assert not dst[e].any(), e


def check_large_routing(T, E, k, seed, scored=True):
    """Routing of many tokens against a stable sort of its own choices, which are checked
    against the scores' order (without a rule the logits'); ties go to the lower index."""
    announce(f"routing T={T} E={E} k={k} scored={scored}")
    g = torch.Generator(device=DEV).manual_seed(seed)
    lg = torch.rand((T, E), device=DEV, generator=g) * 8 - 4
    r = bq.DeviceRouting(T, E, k, 64, DEV)
    for t in (r.topk_idx, r.counts, r.offsets, r.sorted_assign, r.assign_row, r.block_expert, r.block_row, r.n_blocks):
        t.fill_(-7)
    ws = torch.empty(max(256, bq.route_workspace_bytes(T, E, k, 64)), dtype=torch.uint8, device=DEV)
    if scored:
        bq.moe_route_scored(lg, None, bq.ScoreRule("sigmoid"), k, 64, r, ws)
    else:
        bq.moe_route(lg, k, 64, r, ws)
    sync()
    score = (1 / (1 + torch.exp(-lg.double()))).float() if scored else lg
    best = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(r.topk_idx, best.int())
    del lg, score, best
    flat = r.topk_idx.view(-1)
    counts = torch.bincount(flat, minlength=E)
    assert torch.equal(r.counts, counts.int())
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), counts.cumsum(0)])
    assert torch.equal(r.offsets, offsets.int())
    order = torch.sort(flat, stable=True)[1]
    assert torch.equal(r.sorted_assign, order.int())
    assert torch.equal(r.assign_row[order], torch.arange(T * k, device=DEV, dtype=torch.int32))
    blocks = (counts + 63) // 64
    n, start = int(blocks.sum()), blocks.cumsum(0) - blocks
    assert int(r.n_blocks) == n
    e = torch.repeat_interleave(torch.arange(E, device=DEV), blocks)
    row = offsets[e] + 64 * (torch.arange(n, device=DEV) - start[e])
    assert torch.equal(r.block_expert[:n], e.int()) and torch.equal(r.block_row[:n], row.int())
    assert (r.block_expert[n:] == -1).all() and (r.block_row[n:] == -1).all()


def test_scored_routing_of_tokens_beyond_one_launch(large):
    check_large_routing((1 << 26) + 3, 2, 1, 0)


# the selection by waves alone, and with chunk information for the grouping
@pytest.mark.parametrize("E,k", [(2, 1), (4, 4)])
def test_routing_of_tokens_beyond_one_launch(large, E, k):
    check_large_routing((1 << 26) + 3, E, k, 1, scored=False)


def test_router_of_tokens_beyond_one_launch(large):
    T, H = (1 << 28) + 40, 64
    announce(f"router T={T}")
    some = [0, (1 << 24) - 1, 1 << 24, T // 2, T - 1]
    rows = dev(np.random.default_rng(0).normal(size=(len(some), H)), torch.bfloat16)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    x[some] = rows
    w, wg = dev(np.random.default_rng(1).normal(size=(1, H)), torch.bfloat16), torch.ones(H, dtype=torch.bfloat16, device=DEV)
    lg, gate = torch.full((T, 1), 9.0, device=DEV), torch.full((T,), 9.0, device=DEV)
    bq.moe_router(x, w, lg, wg, gate)
    sync()
    want = f64(rows) @ f64(w).T
    within(f64(lg[some]), want, H * 2.0 ** -23 * (np.abs(f64(rows)) @ np.abs(f64(w)).T), "logits")
    # a sigmoid's slope is at most 1/4: a quarter of the sum's error, and of exp's (|z| < 32 steps of 2^-23)
    z = f64(rows).sum(1)
    within(f64(gate[some]), 1 / (1 + np.exp(-z)), H * 2.0 ** -23 * np.abs(f64(rows)).sum(1) + 2.0 ** -20, "gate")
    lg[some], gate[some] = 0, 0.5
    assert not lg.any() and (gate == 0.5).all()


# ---- many tokens: work that grows with them ----

# one round of the sums over workgroups and several, counts of one word and of many
@pytest.mark.parametrize("T,E,k", [(8193, 256, 8), (65537, 2, 1), (33333, 40, 3), (70001, 1000, 8), (300000, 60, 4), (1100000, 1, 1),
                                   (1 << 22, 64, 8)])
def test_scored_routing_of_many_tokens(large, T, E, k):
    check_large_routing(T, E, k, T)


def test_scored_routings_time_follows_its_tokens(large):
    """Sixteen times the tokens take about 15 times as long; where every grouping workgroup sums
    all tokens' counts itself, 118 times."""
    def best(T):
        E, k = 256, 8
        lg = torch.randn((T, E), device=DEV)
        r = bq.DeviceRouting(T, E, k, 64, DEV)
        ws = torch.empty(bq.route_workspace_bytes(T, E, k, 64), dtype=torch.uint8, device=DEV)
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                bq.moe_route_scored(lg, None, bq.ScoreRule("sigmoid"), k, 64, r, ws)
            b.record()
            sync()
            times.append(a.elapsed_time(b))
        return min(times)
    assert best(1 << 20) < 64 * best(1 << 16)


# ---- the layer object's buffers ----

def test_release_gives_the_memory_back(large):
    H, I, I_sh, E, k = 256, 128, 64, 16, 2
    g = np.random.default_rng(8)
    mats = [i8mat(q, s, 1) for q, s in layer_weights(g, E, H, I, I_sh)]
    layer = bq.MoeLayerI8(mats, H, I, I_sh, E, k, DEV)
    x, sx = dev(codes(g, 4000, H), torch.int8), dev(g.random(4000), torch.float32) * 0.02
    lg = dev(g.normal(size=(4000, E)), torch.float32)
    run = lambda T, **kw: layer.forward(x[:T], sx[:T], lg[:T], **kw)["y"].clone()  # noqa: E731
    want = run(70)
    start = torch.cuda.memory_allocated()
    run(4000)
    run(4000, stream=torch.cuda.Stream())   # still on its way when the buffers go
    assert torch.cuda.memory_allocated() - start > 8_000_000
    layer.release(4000)
    assert torch.cuda.memory_allocated() - start < 1_000_000
    layer.release()
    got = run(70)
    sync()
    assert torch.equal(got, want)


def test_block_runs_on_its_tensors_device(monkeypatch):
    """Every launch of the block with the tensors' device as the current one (here the other device
    is only claimed to be current: the test needs no second GPU)."""
    require_gpu()
    H, I, E, k, T = 256, 128, 16, 2, 5
    g = np.random.default_rng(8)
    mats = [i8mat(q, s, 1) for q, s in layer_weights(g, E, H, I, 0)] + [None] * 3
    layer = bq.MoeLayerI8(mats, H, I, 0, E, k, DEV)
    x, r, w = norm_inputs(T, H, 0)
    router = dev(g.normal(size=(E, H)) * H ** -0.5, torch.bfloat16)
    want = layer.forward_block(x, r, w, router)["y"].clone()
    current, seen, run_router = [1], [], bq.moe_router

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *exc):
            current.pop()

    def routed(*args, **kw):
        seen.append(current[-1])
        run_router(*args, **kw)

    monkeypatch.setattr(bq.torch.cuda, "device", Device)
    monkeypatch.setattr(bq, "_current_device", lambda: current[-1])
    monkeypatch.setattr(bq, "moe_router", routed)
    y = layer.forward_block(x, r, w, router)["y"]
    monkeypatch.undo()
    sync()
    assert seen == [0] and current == [1] and torch.equal(y, want)


def test_one_tokens_rows_are_a_permutation_whatever_its_logits(large):
    """NaN of all bits sorts as no expert at all: the selection then repeats the first, and a
    product over the routing must still find a row for each of its assignments."""
    H = I = 64
    E, k = 8, 4
    g = np.random.default_rng(4)
    mats = [i8mat(q, s, 1) for q, s in layer_weights(g, E, H, I, 0)] + [None] * 3
    layer = bq.MoeLayerI8(mats, H, I, 0, E, k, DEV)
    lg = torch.full((1, E), -1, dtype=torch.int32, device=DEV).view(torch.float32)
    lg[0, 5] = 1.0
    r = layer.buffers(1)["routing"]
    r.sorted_assign.fill_(-7)
    layer.forward(dev(codes(g, 1, H), torch.int8), torch.ones(1, device=DEV), lg)
    sync()
    assert int(r.topk_idx.min()) >= 0 and int(r.topk_idx.max()) < E
    assert sorted(r.sorted_assign.tolist()) == list(range(k)) == sorted(r.assign_row.tolist())
    assert [r.assign_row[a].item() for a in r.sorted_assign.tolist()] == list(range(k))


# one launch, chunk information and radix selection; with the layer's counted indices
@pytest.mark.parametrize("T,k", [(1, 4), (3, 8), (70, 8), (70, 6), (20, 20), (70, 20)])
@pytest.mark.parametrize("layer_call", [False, True])
def test_no_expert_twice_whatever_the_logits(T, k, layer_call):
    """Rows of NaN, of all bits and of others, with a few numbers: the chosen experts differ."""
    require_gpu()
    H = I = 64
    E = 24
    g = np.random.default_rng(T + k)
    bits = g.choice(np.array([-1, -1, -1, 0x7FC00000, -0x400000, 0x7F800001], np.int32), (T, E))
    bits[:, 7] = np.float32(1.5).view(np.int32)
    bits[0] = -1
    lg = dev(bits, torch.int32).view(torch.float32)
    mats = [i8mat(q, s, 1) for q, s in layer_weights(g, E, H, I, 0)] + [None] * 3
    layer = bq.MoeLayerI8(mats, H, I, 0, E, k, DEV)
    b = layer.buffers(T)
    r = b["routing"]
    r.sorted_assign.fill_(-7)
    if layer_call:
        layer.forward(dev(codes(g, T, H), torch.int8), torch.ones(T, device=DEV), lg)
    else:
        bq.moe_route(lg, k, r.block_rows, r, b["route_ws"])
    sync()
    idx = r.topk_idx.cpu().numpy()
    assert idx.min() >= 0 and idx.max() < E and all(len(set(row)) == k for row in idx.tolist())
    assert sorted(r.sorted_assign.tolist()) == list(range(T * k)) == sorted(r.assign_row.tolist())


# ---- the layer's routing without a rule ----

ROUTED = [  # T, E, k: one launch, counted indices, and above 32768 assignments; each count of experts a lane;
    # k on both sides of the radix selection
    (16, 256, 8), (17, 256, 8), (512, 256, 8), (4096, 256, 8), (4097, 256, 8), (300, 128, 6), (100, 500, 20), (40, 1000, 10),
    (64, 1000, 64), (33, 64, 16), (33, 64, 17), (2048, 1, 1), (70, 3, 3), (2100, 130, 9), (4096, 600, 8), (32768, 32, 1),
    (32769, 32, 1)]


@pytest.mark.parametrize("T,E,k", ROUTED)
@pytest.mark.parametrize("block_rows", [16, 32, 64])
def test_layers_routing_without_a_rule(T, E, k, block_rows):
    """moe_layer_i8's own routing arrays, with tied logits and tokens that all choose alike."""
    require_gpu()
    announce(f"layer routing T={T} E={E} k={k} rows={block_rows}")
    H = I = 64
    g = np.random.default_rng(T + E)
    rnd = lambda *s: dev(codes(g, *s), torch.int8)  # noqa: E731
    mats = [bq.DeviceI8Mat(rnd(E, 64, 64), torch.full((E, 64), 1e-3, device=DEV)) for _ in range(3)] + [None] * 3
    layer = bq.MoeLayerI8(mats, H, I, 0, E, k, DEV, block_rows=block_rows)
    x, sx = rnd(T, H), torch.full((T,), 0.02, device=DEV)
    lg = g.normal(size=(T, E)).astype(np.float32)
    alike = np.tile(lg[:1], (T, 1))
    tied = np.round(lg)
    ys = []
    for values in (lg, tied, alike, lg):
        got = layer.forward(x, sx, dev(values, torch.float32))
        sync()
        assert_routing_matches(got["routing"].to_host(), values, k, block_rows)
        ys.append(got["y"].clone())
    assert torch.equal(ys[0], ys[3])
