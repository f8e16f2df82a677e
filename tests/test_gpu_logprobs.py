"""moe_logprobs on the GPU against its 64-bit form.

Tolerances.  A thread adds up to V / 512 terms one after another and its sums go through some 20
joins; with the running maximum's rescalings (three roundings, once in 32 values at most) a sum of
positive terms is within (V / 256 + 100) * 2^-24 of itself, exp2 (1 ulp) and its argument's
rounding (|t| * 2^-24 for terms above 2^-24, so 24 of them at most) included.  log S has that much
as an absolute error; z - m, log S and their difference add 2^-22 of |log p| + log V.  The
entropy is log S and the quotient of two such sums, at most log V: twice that share of it."""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_amd as bq
from gpu_cases import DEV, announce, require_gpu
from oracle import serve_oracle

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def sync():
    torch.cuda.synchronize()


def outputs(T, n):
    nan = float("nan")
    o = dict(logprob=torch.full((T,), nan, device=DEV), entropy=torch.full((T,), nan, device=DEV))
    if n:
        o.update(top_idx=torch.full((T, n), -1, dtype=torch.int32, device=DEV),
                 top_logprob=torch.full((T, n), nan, device=DEV))
    return o


def call(z, targets, n, stream=None):
    T, V = z.shape
    o = outputs(T, n)
    nbytes = bq.logprobs_workspace_bytes(T, V, n)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV) if nbytes else None
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    bq.moe_logprobs(z, targets, ws=ws, **o, stream=stream)
    sync()
    return o


def close(got, want, bound, what):
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        off = np.where(same, 0.0, np.abs(got - want))
    bad = ~(off <= bound)
    assert not bad.any(), f"{what} at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


def check(o, z, targets, n, what, rows=None):
    rows = np.arange(len(z)) if rows is None else np.asarray(rows)
    host = z[torch.from_numpy(rows).to(DEV)].float().cpu().numpy()
    lp, ent, idx, top = serve_oracle.logprobs(host, None if targets is None else targets.cpu().numpy()[rows], n)
    V = z.shape[1]
    share = (V / 256 + 100) * 2.0 ** -24

    def bound(v):
        with np.errstate(invalid="ignore"):
            return share + 2.0 ** -22 * (np.where(np.isfinite(v), np.abs(v), 0) + np.log(V))

    if targets is not None:
        close(o["logprob"].double().cpu().numpy()[rows], lp, bound(lp), what + " logprob")
    close(o["entropy"].double().cpu().numpy()[rows], ent, 2 * share * (np.log(V) + 1) + bound(ent), what + " entropy")
    if n:
        assert np.array_equal(o["top_idx"].cpu().numpy()[rows], idx), what
        close(o["top_logprob"].double().cpu().numpy()[rows], top, bound(top), what + " top_logprob")


def rows_of(g, T, V, dtype, spread=3.0):
    return torch.from_numpy((spread * g.standard_normal((T, V))).astype(np.float32)).to(DEV).to(dtype)


def targets_of(g, T, V):
    return torch.from_numpy(g.integers(0, V, T).astype(np.int32)).to(DEV)


# pieces of 16 bytes, whole and cut at both ends (odd rows start inside one), one thread and all,
# one part of a row and several, one row and many
SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (9, 9), (17, 15), (4, 63), (33, 64), (7, 65), (3, 513), (2, 4095), (2, 4097), (5, 8192),
         (1, 12289), (1, 100003), (1, 131072), (3, 40001), (11, 50000), (130, 20011), (1100, 1031), (2100, 515)]


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [0, 1, 20, 64])
def test_rows_of_logits(T, V, dtype, n):
    require_gpu()
    n = min(n, V)
    what = f"logprobs T={T} V={V} {dtype} n={n}"
    announce(what)
    g = np.random.default_rng(T + V)
    z, t = rows_of(g, T, V, dtype), targets_of(g, T, V)
    check(call(z, t, n), z, t, n, what)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift,pad", [(0, 5), (1, 0), (3, 1), (7, 8), (5, 3)])
def test_rows_that_lie_apart(dtype, shift, pad):
    """A head padded to a round vocabulary, or a slice of a wider tensor: rows start anywhere."""
    require_gpu()
    T, V, n = 6, 5003, 7
    announce(f"logprobs strides {dtype} {shift} {pad}")
    g = np.random.default_rng(shift)
    wide = torch.full((T, V + shift + pad), float("inf"), dtype=dtype, device=DEV)   # what lies beside is not read
    z = wide[:, shift:shift + V]
    z.copy_(rows_of(g, T, V, dtype))
    t = targets_of(g, T, V)
    check(call(z, t, n), z, t, n, "apart")
    assert torch.isinf(wide[:, :shift]).all() and torch.isinf(wide[:, shift + V:]).all()


def special_rows(V):
    """Rows where a selection can go wrong, by name."""
    g = np.random.default_rng(4)
    base = 2 * g.standard_normal(V)
    ninf = -np.inf
    few = np.full(V, ninf)
    few[[V // 3, V - 1, 0]] = [1.0, 2.0, 2.0]
    one = np.full(V, ninf)
    one[V // 2] = -4.0
    half = base.copy()
    half[: V // 2] = ninf
    nan, inf2, mixed = base.copy(), base.copy(), np.full(V, ninf)
    nan[V // 5] = np.nan
    inf2[[3, V - 2]] = np.inf
    mixed[V // 4], mixed[V // 7] = np.nan, np.inf
    zeros = np.where(np.arange(V) % 2, 0.0, -0.0)
    spike = base.copy()
    spike[V - 1] = 300.0
    return dict(equal=np.full(V, 1.5), up=np.linspace(-9, 9, V), down=np.linspace(9, -9, V), empty=np.full(V, ninf),
                few=few, one=one, half=half, nan=nan, inf=inf2, mixed=mixed, zeros=zeros, spike=spike,
                lowest=np.full(V, np.float32(-3.3e38)), nans=np.full(V, np.nan), wide=base * 1e30,
                far=np.where(np.arange(V) == 5, 0.0, -200.0))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V,copies", [(37, 1), (1000, 1), (30011, 1), (30011, 70)])
def test_masked_equal_sorted_and_infinite_rows(dtype, V, copies):
    require_gpu()
    announce(f"logprobs special rows V={V} {dtype} x {copies}")
    rows = special_rows(V)
    z = torch.from_numpy(np.stack(list(rows.values())).astype(np.float32)).to(DEV).to(dtype)
    z = z.repeat(copies, 1).contiguous()
    t = torch.full((len(z),), V // 3, dtype=torch.int32, device=DEV)
    check(call(z, t, 20), z, t, 20, "special")
    # an empty row by the written rule
    at = list(rows).index("empty")
    o = call(z, t, 3)
    assert float(o["entropy"][at]) == 0 and o["top_idx"][at].tolist() == [0, 1, 2]
    assert (o["top_logprob"][at] == float("-inf")).all() and float(o["logprob"][at]) == float("-inf")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_largest_values_with_few_threads(dtype):
    """The values above all others lie at one distance from another, in many places, so that a
    few of the threads hold them all."""
    require_gpu()
    T, V, n = 1100, 33000, 12
    announce(f"logprobs few threads {dtype}")
    g = np.random.default_rng(6)
    z = rows_of(g, T, V, dtype, 1.0)
    per = 8 if dtype is BF16 else 4
    at = np.arange(V)
    for row, (threads, step) in enumerate(((9, 512), (11, 512), (12, 512), (300, 512), (11, 256), (11, 1024))):
        large = at[(at // per) % step < threads]
        z[row, torch.from_numpy(large).to(DEV)] = torch.from_numpy(
            (20 + g.random(len(large))).astype(np.float32)).to(DEV).to(dtype)
    t = targets_of(g, T, V)
    check(call(z, t, n), z, t, n, "few threads", rows=list(range(8)) + [1099])


def test_targets_outside_the_row_and_outputs_left_out():
    require_gpu()
    g = np.random.default_rng(2)
    T, V, n = 7, 3000, 4
    z = rows_of(g, T, V, BF16)
    t = torch.tensor([-1, 0, V - 1, V, 2 ** 31 - 1, -2 ** 31, 5], dtype=torch.int32, device=DEV)
    o = call(z, t, n)
    check(o, z, t, n, "targets")
    assert o["logprob"][[0, 3, 4, 5]].tolist() == [0, 0, 0, 0]
    for name in ("logprob", "entropy", "top_idx", "top_logprob"):
        one = torch.zeros_like(o[name])
        bq.moe_logprobs(z, t if name == "logprob" else None, **{name: one})
        sync()
        assert torch.equal(one, o[name])


@pytest.mark.parametrize("T", [2, 60, 1200])
def test_captured_replayed_and_on_another_stream(T):
    require_gpu()
    announce(f"logprobs graph T={T}")
    V, n = 9001, 8
    g = np.random.default_rng(T)
    sets = [(rows_of(g, T, V, BF16), targets_of(g, T, V)) for _ in range(3)]
    want = [call(*s, n) for s in sets]
    z, t = sets[0][0].clone(), sets[0][1].clone()
    o = outputs(T, n)
    nbytes = bq.logprobs_workspace_bytes(T, V, n)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bq.moe_logprobs(z, t, ws=ws, **o)
    for i in (1, 2, 0, 2):
        z.copy_(sets[i][0])
        t.copy_(sets[i][1])
        graph.replay()
        mine = call(*sets[(i + 1) % 3], n)
        assert all(torch.equal(o[k], want[i][k]) and torch.equal(mine[k], want[(i + 1) % 3][k]) for k in o)
    side = call(*sets[1], n, stream=torch.cuda.Stream())
    assert all(torch.equal(side[k], want[1][k]) for k in side)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_special_rows_in_parts(dtype):
    """Rows that are split over workgroups and joined, also where they start inside a piece."""
    require_gpu()
    announce(f"logprobs special rows in parts {dtype}")
    V = 70011
    rows = special_rows(V)
    wide = torch.full((len(rows), V + 6), float("inf"), dtype=dtype, device=DEV)
    z = wide[:, 3:3 + V]
    z.copy_(torch.from_numpy(np.stack(list(rows.values())).astype(np.float32)))
    t = torch.full((len(z),), V // 3, dtype=torch.int32, device=DEV)
    for n in (1, 20, 64):
        check(call(z, t, n), z, t, n, "special in parts")
    # the best tokens all in one part, and at its ends
    g = np.random.default_rng(12)
    z = rows_of(g, 5, 200003, dtype, 1.0)
    z[0, :40] += 30
    z[1, -40:] += 30
    z[2, 100000:100040] += 30
    z[3, ::4001] += 30
    t = targets_of(g, 5, 200003)
    check(call(z, t, 30), z, t, 30, "parts")


def test_parts_captured_and_on_two_streams():
    require_gpu()
    announce("logprobs in parts, captured and on two streams")
    T, V, n = 3, 80001, 9
    g = np.random.default_rng(3)
    sets = [(rows_of(g, T, V, BF16), targets_of(g, T, V)) for _ in range(2)]
    want = [call(*s, n) for s in sets]
    z, t, o = sets[0][0].clone(), sets[0][1].clone(), outputs(T, n)
    wss = [torch.zeros(bq.logprobs_workspace_bytes(T, V, n), dtype=torch.uint8, device=DEV) for _ in range(3)]
    assert wss[0].numel()
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bq.moe_logprobs(z, t, ws=wss[0], **o)
    for i in (1, 0, 1):
        z.copy_(sets[i][0])
        t.copy_(sets[i][1])
        graph.replay()
        mine = call(*sets[1 - i], n)
        assert all(torch.equal(o[k], want[i][k]) and torch.equal(mine[k], want[1 - i][k]) for k in o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [outputs(T, n) for _ in range(12)]
    sync()
    for i, out in enumerate(outs):
        bq.moe_logprobs(*sets[i % 2], ws=wss[1 + i % 2], **out, stream=streams[i % 2])
    sync()
    assert all(torch.equal(out[k], want[i % 2][k]) for i, out in enumerate(outs) for k in out)


def test_rows_far_into_a_large_tensor():
    """Rows whose offsets pass 2^32 bytes."""
    require_gpu()
    announce("logprobs far rows")
    V, T = 1 << 20, 2100
    z = torch.zeros((T, V), dtype=BF16, device=DEV)
    z[T - 1, V - 3] = 4.0
    z[T - 1, 77] = 4.0
    t = torch.full((T,), 77, dtype=torch.int32, device=DEV)
    o = call(z, t, 2)
    check(o, z, t, 2, "far", rows=[0, T - 1])


def test_the_head_and_its_log_probabilities():
    """The operators in a run, as a step that serves several requests has them: norm, a projection
    with each request's adapter, norm, the layer of a few tokens, the head and the log probabilities; each
    stage against its form over the stage before's own output."""
    require_gpu()
    announce("a step of several requests")
    import test_gpu_batch as tb
    import test_gpu_i8 as ti
    import test_gpu_lora as tl
    from oracle import route_topk
    T, H, I, I_sh, E, k, V, R, n = 13, 256, 128, 64, 16, 4, 4001, 16, 5
    g = np.random.default_rng(1)
    x, res, w = ti.norm_inputs(T, H, 5)
    s, y = (torch.empty((T, H), dtype=BF16, device=DEV) for _ in range(2))
    q, qs = torch.empty((T, H), dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    bq.moe_norm_i8(x, res, w, ti.EPS, s, y, q, qs)
    h, args = tl.make(g, T, H, H, R, n, tl.pattern(g, T, n, "rows"), True)
    proj = torch.empty((T, H), dtype=BF16, device=DEV)
    bq.moe_linear_lora_i8(q, qs, args["w"], args["adapters"], args["adapter"], proj, tl.workspace(T, H, H, R))
    normed, q2, qs2 = torch.empty_like(y), torch.empty_like(q), torch.empty_like(qs)
    bq.moe_norm_i8(proj, s, w, ti.EPS, None, normed, q2, qs2)
    router = ti.dev(g.normal(size=(E, H)) * H ** -0.5, BF16)
    lg = torch.empty((T, E), device=DEV)
    bq.moe_router(normed, router, lg)
    host = tb.host_mats(g, E, H, I, I_sh)
    layer = bq.MoeLayer.from_device(tb.device_mats(host, bq.LAYOUT_TILES_SB), H, I, I_sh, E, k, DEV)
    got = layer.decode_batch(normed, lg)
    bq.moe_quant_i8(got["y"], q2, qs2)
    head = bq.DeviceI8Mat.from_bf16(ti.dev(g.normal(size=(1, V, H)), BF16))
    z = torch.empty((T, V), dtype=BF16, device=DEV)
    bq.moe_linear_i8(q2, qs2, head, z)
    t = targets_of(g, T, V)
    o = call(z, t, 5)
    h.update(a=q.cpu().numpy(), sa=qs.cpu().numpy())
    tl.check(proj, h, "projection")
    idx, wgt = route_topk(lg.cpu().numpy(), k)
    tb.check_y(got["y"], serve_oracle.batch_layer(tb.host_of(normed), idx, wgt, host[:3], host[3:], None), "layer")
    check(o, z, t, 5, "log probabilities")
