"""moe_decode_batch_q4 (1 to 64 tokens through the 4-bit layer) on the GPU against its 64-bit form.

Tolerances.  y is the nearest bf16 to an fp32 value: half a step is 2^-8 of it.  That value's own
error: h has two bf16, 2^-16 of each; sums of K products of bf16 values (each product exact) make
one rounding of 2^-24 of the running sum for a term, independent of each other, and the
magnitudes' sum is at most about sqrt(K) times the sum for terms of random sign: sqrt(K) * sqrt(K)
* 2^-24, 2^-12 at K 4096, as a root mean square of a row; silu has 1 ulp in exp2 and the reciprocal
each, below that.  An element may be 4 root mean squares off: 2^-10 of the row's.  Rows whose
values cancel are not made here.
The selection is exact, its weights have 1e-6 as in the routing call's own tests."""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_amd as bq
import oracle
from gpu_cases import DEV, announce, require_gpu
from oracle import i8_oracle, serve_oracle
from workload import draw_qmat, f32_to_bf16_bits

pytestmark = pytest.mark.gpu

HALF, ROW = 2.0 ** -8, 2.0 ** -10


def sync():
    torch.cuda.synchronize()


def host_mats(g, E, H, I, I_sh):
    shapes = [(E, I, H), (E, I, H), (E, H, I)] + ([(1, I_sh, H), (1, I_sh, H), (1, H, I_sh)] if I_sh else [])
    return [draw_qmat(g, *s) for s in shapes]


def device_mats(host, layout):
    mats = [bq.DeviceQMat.from_host(m, DEV) for m in host]
    if layout != bq.LAYOUT_ROWS:
        mats = bq.prepacked_mats(mats + [None] * (6 - len(mats)), pack_scales=layout == bq.LAYOUT_TILES_SB)
    return tuple(mats) + (None,) * (6 - len(mats))


def inputs(g, T, H, E):
    x = bq.bf16_from_bits(f32_to_bf16_bits(g.standard_normal((T, H), dtype=np.float32)), DEV)
    return x, torch.from_numpy(g.standard_normal((T, E), dtype=np.float32)).to(DEV)


def host_of(x):
    return x.double().cpu().numpy()


def check_y(y, want, what, K=4096):
    got = host_of(y)
    rms = np.sqrt((want ** 2).mean(1, keepdims=True))
    bound = HALF * np.abs(want) + ROW * max(1, K / 4096) * rms
    worst = np.unravel_index(np.argmax(np.abs(got - want) - bound), got.shape)
    assert (np.abs(got - want) <= bound).all(), f"{what} at {worst}: {got[worst]} for {want[worst]}"


def check_call(T, H, I, I_sh, E, k, layout, rule=None, gated=False, seed=0, logits=None):
    what = f"batch T={T} H={H} I={I} I_sh={I_sh} E={E} k={k} layout={layout} rule={rule} gated={gated}"
    announce(what)
    g = np.random.default_rng(seed + T + H + I)
    host = host_mats(g, E, H, I, I_sh)
    mats = device_mats(host, layout)
    x, lg = inputs(g, T, H, E)
    lg = lg if logits is None else torch.from_numpy(logits.astype(np.float32)).to(DEV)
    bias = torch.from_numpy((0.05 * g.standard_normal(E)).astype(np.float32)).to(DEV) if rule else None
    gate = torch.from_numpy(g.uniform(0.1, 0.9, T).astype(np.float32)).to(DEV) if gated else None
    ws = torch.full((bq.decode_batch_workspace_bytes(T, H, I, I_sh, E, k),), 0xFF, dtype=torch.uint8, device=DEV)
    y = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    idx = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), float("nan"), device=DEV)
    dev_rule = None if rule is None else bq.ScoreRule(**rule)
    bq.moe_decode_batch_q4(x, lg, bias, dev_rule, gate, I, I_sh, k, *mats, y, ws, idx, w)
    sync()
    if rule is None:
        want_idx, want_w = oracle.route_topk(lg.cpu().numpy(), k)
    else:
        r = dict(rule, sigmoid=rule.get("score") == "sigmoid", top2=rule.get("group_score", "top2") == "top2")
        r.pop("score", None), r.pop("group_score", None)
        want_idx, want_w = i8_oracle.route_scored(lg.cpu().numpy(), bias.cpu().numpy(), k, **r)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    assert np.max(np.abs(w.double().cpu().numpy() - want_w)) <= 1e-6 * max(1.0, np.abs(want_w).max())
    want = serve_oracle.batch_layer(host_of(x), want_idx, want_w, host[:3], host[3:] if I_sh else None,
                                    None if gate is None else gate.cpu().numpy())
    check_y(y, want, what, max(H, I, I_sh))
    # without the selection's outputs, with another workspace: bit for bit
    y2, ws2 = torch.empty_like(y), torch.zeros_like(ws)
    bq.moe_decode_batch_q4(x, lg, bias, dev_rule, gate, I, I_sh, k, *mats, y2, ws2)
    sync()
    assert torch.equal(y, y2)


# on both sides of every change of form: 8, 16 and 32 tokens, 32 and 128 chosen experts, widths of
# an odd number of 64s, one expert, all experts, many per token
SHAPES = [
    (1, 64, 64, 0, 1, 1), (1, 256, 128, 64, 16, 4), (2, 2048, 512, 512, 64, 8), (3, 192, 64, 320, 8, 3),
    (4, 320, 192, 0, 40, 8), (7, 448, 576, 128, 60, 4), (8, 128, 64, 64, 300, 16), (9, 128, 64, 64, 300, 16),
    (8, 256, 320, 0, 3, 3), (15, 576, 128, 192, 16, 2), (16, 256, 128, 64, 60, 9), (17, 256, 128, 64, 60, 9),
    (16, 1024, 256, 0, 6, 6), (32, 192, 128, 64, 24, 4), (33, 192, 128, 64, 24, 4), (48, 64, 192, 0, 130, 3),
    (64, 256, 64, 128, 512, 5), (64, 128, 64, 0, 1000, 2), (64, 128, 128, 64, 2, 1), (64, 64, 64, 64, 64, 64),
    (5, 128, 64, 0, 70, 20), (20, 128, 64, 0, 70, 20), (63, 384, 1088, 1152, 3, 2)]


@pytest.mark.parametrize("T,H,I,I_sh,E,k", SHAPES)
@pytest.mark.parametrize("layout", [bq.LAYOUT_ROWS, bq.LAYOUT_TILES, bq.LAYOUT_TILES_SB])
def test_layer_of_a_few_tokens(T, H, I, I_sh, E, k, layout):
    require_gpu()
    check_call(T, H, I, I_sh, E, k, layout, gated=bool(I_sh) and T % 2 == 0)


# x or h of an entry's tokens in more than one part, the last of half a chunk; entries of 16 and more
@pytest.mark.parametrize("T,H,I,I_sh,E,k", [
    (1, 4160, 64, 0, 3, 2), (6, 4160, 64, 64, 3, 2), (8, 8192, 64, 64, 3, 1), (14, 8256, 64, 128, 5, 2),
    (64, 4160, 128, 64, 6, 2), (40, 8192, 64, 0, 2, 2), (12, 128, 4160, 64, 4, 2), (50, 64, 4160, 2112, 3, 2),
    (16, 192, 128, 4224, 3, 1)])
@pytest.mark.parametrize("layout", [bq.LAYOUT_ROWS, bq.LAYOUT_TILES_SB])
def test_operands_that_do_not_fit_at_once(T, H, I, I_sh, E, k, layout):
    require_gpu()
    check_call(T, H, I, I_sh, E, k, layout)


def test_scales_at_odd_places():
    """Scales and biases of rows may start at any multiple of 2 bytes."""
    require_gpu()
    announce("batch, scales 2 bytes into an allocation")
    for T in (3, 20):
        H, I, I_sh, E, k = 256, 128, 64, 10, 2
        g = np.random.default_rng(T)
        mats = device_mats(host_mats(g, E, H, I, I_sh), bq.LAYOUT_ROWS)
        x, lg = inputs(g, T, H, E)
        want = bq.MoeLayer.from_device(mats, H, I, I_sh, E, k, DEV).decode_batch(x, lg)["y"].clone()
        moved = []
        for m in mats:
            parts = []
            for t in (m.scales, m.biases):
                room = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
                room[1:] = t.reshape(-1)
                parts.append(room[1:].view(t.shape))
            moved.append(bq.DeviceQMat(m.codes, *parts, m.layout))
        y = bq.MoeLayer.from_device(tuple(moved), H, I, I_sh, E, k, DEV).decode_batch(x, lg)["y"]
        sync()
        assert torch.equal(y, want)


@pytest.mark.parametrize("T", [1, 3, 8, 9, 20, 64])
@pytest.mark.parametrize("rule", [
    dict(score="softmax", renormalise=False, scale=16.0),
    dict(score="sigmoid", n_groups=8, topk_groups=4, scale=2.5),
    dict(score="softmax", n_groups=6, topk_groups=2, group_score="max")])
def test_scored_selection(T, rule):
    require_gpu()
    check_call(T, 256, 128, 64, 48, 6, bq.LAYOUT_TILES_SB, rule=rule, gated=True)


@pytest.mark.parametrize("T", [2, 8, 16, 40, 64])
def test_all_tokens_choose_alike_and_ties_go_to_the_lowest(T):
    require_gpu()
    same = np.zeros((T, 80))
    check_call(T, 256, 192, 64, 80, 5, bq.LAYOUT_TILES_SB, logits=same)   # experts 0 .. 4
    one = np.random.default_rng(1).normal(size=(T, 80))
    one[:, 79] = 9.0   # the last expert is everyone's first
    check_call(T, 256, 192, 0, 80, 5, bq.LAYOUT_TILES, logits=one)


def test_masked_logits_under_a_rule():
    """Experts switched off, and padded tokens whose row is -inf alone: weight 0, y the shared
    expert's alone; other tokens are what they are without them."""
    require_gpu()
    T, H, I, I_sh, E, k = 6, 128, 64, 64, 32, 4
    g = np.random.default_rng(5)
    host = host_mats(g, E, H, I, I_sh)
    mats = device_mats(host, bq.LAYOUT_TILES_SB)
    x, lg = inputs(g, T, H, E)
    lg[:, 3:9] = float("-inf")
    lg[4] = float("-inf")
    rule = bq.ScoreRule(renormalise=True)
    layer = bq.MoeLayer.from_device(mats, H, I, I_sh, E, k, DEV)
    b = layer.decode_batch(x, lg, rule=rule)
    sync()
    idx, w = i8_oracle.route_scored(lg.cpu().numpy(), None, k)
    assert np.array_equal(b["topk_idx"].cpu().numpy(), idx) and not b["topk_w"][4].any()
    check_y(b["y"], serve_oracle.batch_layer(host_of(x), idx, w, host[:3], host[3:], None), "masked")


def test_a_nan_stays_with_its_token():
    require_gpu()
    for T in (5, 24, 50):
        announce(f"batch NaN T={T}")
        g = np.random.default_rng(T)
        mats = device_mats(host_mats(g, 8, 128, 64, 64), bq.LAYOUT_TILES_SB)
        x, lg = inputs(g, T, 128, 8)
        layer = bq.MoeLayer.from_device(mats, 128, 64, 64, 8, 3, DEV)
        clean = layer.decode_batch(x, lg)["y"].clone()
        x2 = x.clone()
        x2[T // 2, 77] = float("nan")
        x2[1, 5] = float("inf")
        y = layer.decode_batch(x2, lg)["y"]
        sync()
        assert y[T // 2].isnan().all() and not y[1].isfinite().any()
        keep = [t for t in range(T) if t not in (1, T // 2)]
        assert torch.equal(y[keep], clean[keep])


def test_one_token_matches_the_single_token_call():
    """The same function as moe_decode_q4 up to that call's roundings: h to bf16 there (2^-8 of
    each value, independent: 2^-9 of a row's root mean square), weights not rounded there (2^-9 of
    each weight at most, 2^-10 as a root mean square, in both products of a sum)."""
    require_gpu()
    announce("batch against decode, one token")
    H, I, I_sh, E, k = 512, 256, 128, 32, 4
    g = np.random.default_rng(3)
    mats = device_mats(host_mats(g, E, H, I, I_sh), bq.LAYOUT_TILES)
    x, lg = inputs(g, 1, H, E)
    layer = bq.MoeLayer.from_device(mats, H, I, I_sh, E, k, DEV)
    y = layer.decode_batch(x, lg)["y"]
    y1 = torch.empty_like(y)
    layer.decode(x, lg, y1)
    sync()
    d = (y.double() - y1.double())[0].cpu().numpy()
    rms = float(y1.double().square().mean().sqrt())
    assert np.abs(d).max() <= 2 * HALF * np.abs(host_of(y1)).max() + 4 * rms * 2.0 ** -7


@pytest.mark.parametrize("T", [3, 12, 40])
def test_captured_replayed_and_on_another_stream(T):
    require_gpu()
    announce(f"batch graph T={T}")
    H, I, I_sh, E, k = 256, 128, 64, 24, 4
    g = np.random.default_rng(T)
    mats = device_mats(host_mats(g, E, H, I, I_sh), bq.LAYOUT_TILES_SB)
    layer = bq.MoeLayer.from_device(mats, H, I, I_sh, E, k, DEV)
    other = bq.MoeLayer.from_device(mats, H, I, I_sh, E, k, DEV)
    sets = [inputs(g, T, H, E) for _ in range(3)]
    want = [other.decode_batch(*s)["y"].clone() for s in sets]
    x, lg = sets[0][0].clone(), sets[0][1].clone()
    layer.decode_batch(x, lg)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = layer.decode_batch(x, lg)
    for i in (1, 2, 0, 1):
        x.copy_(sets[i][0])
        lg.copy_(sets[i][1])
        graph.replay()
        mine = other.decode_batch(*sets[(i + 1) % 3])["y"]   # eager work of another object in between
        sync()
        assert torch.equal(b["y"], want[i]) and torch.equal(mine, want[(i + 1) % 3])
    side = torch.cuda.Stream()
    fresh = bq.MoeLayer.from_device(mats, H, I, I_sh, E, k, DEV)
    y = fresh.decode_batch(*sets[2], stream=side)["y"]
    side.synchronize()
    assert torch.equal(y, want[2])


def test_two_streams_with_an_object_each():
    require_gpu()
    announce("batch on two streams")
    T, H, I, I_sh, E, k = 10, 512, 128, 64, 40, 4
    g = np.random.default_rng(2)
    mats = device_mats(host_mats(g, E, H, I, I_sh), bq.LAYOUT_TILES_SB)
    layers = [bq.MoeLayer.from_device(mats, H, I, I_sh, E, k, DEV) for _ in range(2)]
    sets = [inputs(g, T, H, E) for _ in range(2)]
    want = [layers[0].decode_batch(*s)["y"].clone() for s in sets]
    sync()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(want[0]) for _ in range(20)]
    for i, o in enumerate(outs):
        layers[i % 2].decode_batch(*sets[i % 2], out=o, stream=streams[i % 2])
    sync()
    assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(outs))


def test_rows_behind_the_output_stay():
    require_gpu()
    T, H, I, E, k = 11, 128, 64, 8, 2
    g = np.random.default_rng(8)
    mats = device_mats(host_mats(g, E, H, I, 0), bq.LAYOUT_ROWS)
    x, lg = inputs(g, T, H, E)
    ws = torch.empty(bq.decode_batch_workspace_bytes(T, H, I, 0, E, k) + 256, dtype=torch.uint8, device=DEV)
    ws[-256:] = 0x5A
    room = torch.full((T + 3, H), 7.0, dtype=torch.bfloat16, device=DEV)
    bq.moe_decode_batch_q4(x, lg, None, None, None, I, 0, k, *mats, room[1:T + 1], ws)
    sync()
    assert (room[0] == 7).all() and (room[T + 1:] == 7).all() and (ws[-256:] == 0x5A).all()
    assert not (room[1:T + 1] == 7).all()


def test_the_layers_other_matrices_are_taken_up():
    """The object checks its matrix sets once; sets that are replaced are checked and used."""
    require_gpu()
    T, H, I, E, k = 4, 128, 64, 8, 2
    g = np.random.default_rng(8)
    a, b = (device_mats(host_mats(g, E, H, I, 0), bq.LAYOUT_ROWS) for _ in range(2))
    x, lg = inputs(g, T, H, E)
    layer = bq.MoeLayer.from_device(a, H, I, 0, E, k, DEV)
    first = layer.decode_batch(x, lg)["y"].clone()
    layer.gate, layer.up, layer.down = b[:3]
    second = layer.decode_batch(x, lg)["y"].clone()
    want = bq.MoeLayer.from_device(b, H, I, 0, E, k, DEV).decode_batch(x, lg)["y"]
    sync()
    assert torch.equal(second, want) and not torch.equal(first, second)
    layer.down = device_mats(host_mats(g, E, H, 2 * I, 0), bq.LAYOUT_ROWS)[2]
    with pytest.raises(ValueError):
        layer.decode_batch(x, lg)
