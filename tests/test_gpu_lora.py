"""moe_linear_lora_i8 (a projection with an adapter for each row) on the GPU against its 64-bit form.

Tolerances.  out is the nearest bf16 to an fp32 value: half a step is 2^-8 of it.  That value: the
codes' sum is exact, int -> fp32 and two products make 3 * 2^-24 of it, the additions of the
adapters' part as much again; an adapter's first product sums K exact products in fp32 (at most
K roundings), its scale and a_scale are two, it is used to 16 bits (2^-16), and the second sums
2 * rank products: all of them shares of the sum of the products' magnitudes."""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_amd as bq
from gpu_cases import DEV, announce, require_gpu
from oracle import serve_oracle

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


def sync():
    torch.cuda.synchronize()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def make(g, M, N, K, R, n, of, tiles):
    """Host arrays, and what the call takes of them."""
    h = dict(a=g.integers(-127, 128, (M, K)).astype(np.int8), sa=g.uniform(0.005, 0.02, M).astype(np.float32),
             w=g.integers(-127, 128, (N, K)).astype(np.int8), sw=(g.uniform(0.5, 1, N) / 127 * K ** -0.5).astype(np.float32),
             s=g.uniform(-2, 2, n).astype(np.float32), of=np.asarray(of, dtype=np.int32))
    A = dev(g.normal(size=(n, R, K)) * K ** -0.5, torch.bfloat16)
    B = dev(g.normal(size=(n, N, R)) * R ** -0.5, torch.bfloat16)
    h["A"], h["B"] = A.float().cpu().numpy(), B.float().cpu().numpy()
    mat = bq.DeviceI8Mat(dev(h["w"], torch.int8)[None], dev(h["sw"], torch.float32)[None])
    return h, dict(a=dev(h["a"], torch.int8), a_scale=dev(h["sa"], torch.float32), w=mat.prepacked() if tiles else mat,
                   adapters=bq.DeviceAdapters(A, B, dev(h["s"], torch.float32)), adapter=dev(h["of"], torch.int32))


def workspace(M, N, K, R):
    return torch.full((bq.linear_lora_i8_workspace_bytes(M, N, K, R),), 0xFF, dtype=torch.uint8, device=DEV)


def check(out, h, what):
    want, size = serve_oracle.linear_lora(h["a"], h["sa"], h["w"], h["sw"], h["A"], h["B"], h["s"], h["of"])
    K, R = h["a"].shape[1], h["A"].shape[1]
    off = size * (2.0 ** -16 + (K + 2 * R + 16) * 2.0 ** -24) + 8 * 2.0 ** -24 * (np.abs(want) + size)
    got = out.double().cpu().numpy()
    err, bound = np.abs(got - want), HALF * (np.abs(want) + off) + off
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), f"{what} at {worst}: {got[worst]} for {want[worst]}, bound {bound[worst]}"


def pattern(g, M, n, kind):
    if kind == "one":
        return np.full(M, n - 1)
    if kind == "rows":
        return g.integers(-1, n, M)
    cut = np.sort(g.integers(0, M + 1, n))
    return g.permutation(n + 1)[(np.arange(M)[:, None] >= cut).sum(1)] - 1


# a size for every form of the dense product, and one on each side of the changes of the adapters' forms
SIZES = [
    (1, 16, 64), (1, 4096, 2048), (2, 45, 192), (5, 1001, 704), (15, 160, 1024), (16, 64, 128), (17, 33, 64), (31, 512, 576),
    (48, 2048, 128), (64, 4096, 192), (128, 4096, 64), (128, 4001, 192), (200, 4096, 128), (500, 4096, 64),
    (333, 1001, 256), (1000, 4096, 128), (1023, 48, 192), (1024, 48, 192), (1100, 70, 1088), (2048, 4096, 64),
    (4096, 4096, 64)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("R,n,kind", [(16, 4, "runs"), (8, 64, "rows"), (40, 3, "one"), (128, 7, "rows")])
def test_projection_with_adapters(M, N, K, R, n, kind):
    require_gpu()
    what = f"lora M={M} N={N} K={K} R={R} n={n} {kind}"
    announce(what)
    g = np.random.default_rng(M + N + K + R)
    h, args = make(g, M, N, K, R, n, pattern(g, M, n, kind), N % 16 == 0)
    room = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = room[:M * N].view(M, N)
    bq.moe_linear_lora_i8(**args, out=out, ws=workspace(M, N, K, R))
    sync()
    check(out, h, what)
    assert (room[M * N:] == 7).all()
    # again over another workspace's bits: the same values
    again = torch.empty_like(out)
    bq.moe_linear_lora_i8(**args, out=again, ws=torch.zeros_like(workspace(M, N, K, R)))
    # rows without an adapter have the plain product's values
    plain = torch.empty_like(out)
    bq.moe_linear_i8(args["a"], args["a_scale"], args["w"], plain)
    sync()
    none = dev(h["of"], torch.int64) < 0
    assert torch.equal(out, again) and torch.equal(out[none], plain[none])


@pytest.mark.parametrize("R", [8, 16, 24, 32, 56, 64, 72, 120, 128])
@pytest.mark.parametrize("M,N,K", [(7, 96, 640), (96, 4096, 128), (1030, 300, 320)])
def test_ranks(M, N, K, R):
    require_gpu()
    what = f"lora ranks M={M} N={N} K={K} R={R}"
    announce(what)
    g = np.random.default_rng(R + M)
    h, args = make(g, M, N, K, R, 5, pattern(g, M, 5, "rows"), N % 16 == 0)
    out = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    bq.moe_linear_lora_i8(**args, out=out, ws=workspace(M, N, K, R))
    sync()
    check(out, h, what)


@pytest.mark.parametrize("M", [4, 40, 1200])
def test_rows_without_an_adapter(M):
    """Numbers outside 0 .. n - 1, the largest and smallest among them, are no adapter; a call may
    have none at all."""
    require_gpu()
    announce(f"lora none M={M}")
    g = np.random.default_rng(M)
    of = g.choice([-1, 3, -2 ** 31, 2 ** 31 - 1, 1 << 20], M)
    h, args = make(g, M, 160, 256, 16, 3, of, True)
    out, plain = (torch.full((M, 160), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = workspace(M, 160, 256, 16)
    bq.moe_linear_lora_i8(**args, out=out, ws=ws)
    bq.moe_linear_i8(args["a"], args["a_scale"], args["w"], plain)
    sync()
    assert torch.equal(out, plain)
    h["of"][M // 2] = 2
    args["adapter"][M // 2] = 2
    bq.moe_linear_lora_i8(**args, out=out, ws=ws)
    sync()
    check(out, h, "one row with an adapter")


@pytest.mark.parametrize("M,N", [(6, 64), (64, 4096), (300, 1000), (2048, 512)])
def test_an_adapters_infinities_stay_with_its_rows(M, N):
    require_gpu()
    announce(f"lora NaN M={M} N={N}")
    g = np.random.default_rng(M)
    of = pattern(g, M, 4, "rows")
    of[:5] = [0, 1, 2, 3, -1]
    h, args = make(g, M, N, 128, 16, 4, of, N % 16 == 0)
    out, bad = (torch.empty((M, N), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = workspace(M, N, 128, 16)
    bq.moe_linear_lora_i8(**args, out=out, ws=ws)
    args["adapters"].a[1, 3, 7] = float("nan")
    args["adapters"].b[2, :, 5] = float("inf")
    args["a_scale"][0] = float("nan")
    bq.moe_linear_lora_i8(**args, out=bad, ws=ws)
    sync()
    of = dev(h["of"], torch.int64)
    keep = (of != 1) & (of != 2)
    keep[0] = False
    assert torch.equal(out[keep], bad[keep])
    assert bad[of == 1].isnan().all() and not bad[of == 2].isfinite().any() and bad[0].isnan().all()


@pytest.mark.parametrize("M", [3, 50, 1500])
def test_captured_replayed_and_on_another_stream(M):
    require_gpu()
    announce(f"lora graph M={M}")
    N, K, R, n = 256, 384, 24, 6
    g = np.random.default_rng(M)
    h, args = make(g, M, N, K, R, n, pattern(g, M, n, "runs"), True)
    sets = [(args["a"].clone(), dev(pattern(g, M, n, "rows"), torch.int32)) for _ in range(3)]
    sets[1][0].neg_()
    want = []
    ws = workspace(M, N, K, R)
    for a, of in sets:
        o = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
        bq.moe_linear_lora_i8(**dict(args, a=a, adapter=of), out=o, ws=ws)
        want.append(o)
    out, ws2 = torch.empty_like(want[0]), workspace(M, N, K, R)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bq.moe_linear_lora_i8(**args, out=out, ws=ws2)
    for i in (0, 1, 2, 1):
        args["a"].copy_(sets[i][0])
        args["adapter"].copy_(sets[i][1])
        graph.replay()
        o = torch.empty_like(out)   # eager work of another workspace in between
        bq.moe_linear_lora_i8(**dict(args, a=sets[(i + 1) % 3][0], adapter=sets[(i + 1) % 3][1]), out=o, ws=ws)
        sync()
        assert torch.equal(out, want[i]) and torch.equal(o, want[(i + 1) % 3])
    side = torch.cuda.Stream()
    o = torch.empty_like(out)
    sync()
    bq.moe_linear_lora_i8(**dict(args, a=sets[2][0], adapter=sets[2][1]), out=o, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(o, want[2])


@pytest.mark.parametrize("M,N,K,R,n,kind", [
    (2100, 256, 512, 64, 40, "rows"), (2100, 256, 512, 64, 40, "runs"), (2100, 80, 512, 64, 40, "one"),
    (2100, 45, 512, 64, 40, "none"), (9001, 64, 128, 64, 30, "rows"), (9001, 33, 128, 72, 3000, "rows"),
    (2050, 64, 512, 64, 5000, "rows")])
def test_rows_in_order_of_their_adapters(M, N, K, R, n, kind):
    """Enough rows and adapters that rows are put in order first, more adapters than that takes, more
    rows than one round of it, no row with an adapter; captured, with other adapters at each replay."""
    require_gpu()
    what = f"lora in order M={M} N={N} K={K} R={R} n={n} {kind}"
    announce(what)
    g = np.random.default_rng(M + n)
    of = np.full(M, -1) if kind == "none" else pattern(g, M, n, kind)
    h, args = make(g, M, N, K, R, n, of, N % 16 == 0)
    out = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = workspace(M, N, K, R)
    bq.moe_linear_lora_i8(**args, out=out[:M], ws=ws)
    sync()
    check(out[:M], h, what)
    assert (out[M:] == 7).all()
    first = out[:M].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bq.moe_linear_lora_i8(**args, out=out[:M], ws=ws)
    other = dev(pattern(g, M, n, "rows"), torch.int32)
    want = torch.empty_like(first)
    bq.moe_linear_lora_i8(**dict(args, adapter=other), out=want, ws=workspace(M, N, K, R))
    mine = args["adapter"].clone()
    for a, w in ((other, want), (mine, first), (other, want)):
        args["adapter"].copy_(a)
        graph.replay()
        sync()
        assert torch.equal(out[:M], w)


@pytest.mark.parametrize("M", [2, 60, 1300])
def test_two_streams_with_a_workspace_each(M):
    """The same adapters and weights from two streams at once."""
    require_gpu()
    announce(f"lora on two streams M={M}")
    N, K, R, n = 300, 512, 16, 9
    g = np.random.default_rng(M)
    h, args = make(g, M, N, K, R, n, pattern(g, M, n, "rows"), False)
    calls = [args, dict(args, adapter=dev(pattern(g, M, n, "runs"), torch.int32))]
    wss = [workspace(M, N, K, R) for _ in calls]
    want = [torch.empty((M, N), dtype=torch.bfloat16, device=DEV) for _ in calls]
    for c, o, ws in zip(calls, want, wss):
        bq.moe_linear_lora_i8(**c, out=o, ws=ws)
    sync()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [torch.empty_like(want[0]) for _ in range(16)]
    sync()
    for i, o in enumerate(outs):
        bq.moe_linear_lora_i8(**calls[i % 2], out=o, ws=wss[i % 2], stream=streams[i % 2])
    sync()
    assert all(torch.equal(o, want[i % 2]) for i, o in enumerate(outs))


def test_an_adapter_is_exchanged_in_place():
    require_gpu()
    g = np.random.default_rng(0)
    h, args = make(g, 9, 64, 128, 8, 3, [0, 1, 2] * 3, True)
    out = torch.empty((9, 64), dtype=torch.bfloat16, device=DEV)
    ws = workspace(9, 64, 128, 8)
    bq.moe_linear_lora_i8(**args, out=out, ws=ws)
    ad = args["adapters"]
    ad.a[1].copy_(ad.a[0] * 2)
    ad.b[1].copy_(ad.b[2])
    ad.scales[1] = 3.0
    h["A"][1], h["B"][1], h["s"][1] = 2 * h["A"][0], h["B"][2], 3.0
    bq.moe_linear_lora_i8(**args, out=out, ws=ws)
    sync()
    check(out, h, "exchanged")
