"""moe_linear_lora_i8 in the dense product's tile forms: their steady loop followed by the adapters,
rows just past a tile, and rows in order of their adapters.  Tolerances as in test_gpu_lora."""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_amd as bq
import test_gpu_lora as tl
from gpu_cases import DEV, announce, require_gpu

pytestmark = pytest.mark.gpu


def check_rows(out, h, rows, what):
    """The given rows against the 64-bit form."""
    part = dict(h, a=h["a"][rows], sa=h["sa"][rows], of=h["of"][rows])
    tl.check(out[torch.from_numpy(np.asarray(rows)).to(DEV)], part, what)


def run_case(M, N, K, R, n, kind, what):
    announce(what)
    g = np.random.default_rng(M + N + K + R)
    of = tl.pattern(g, M, n, kind)
    of[[0, M // 2]] = -1   # rows without an adapter, also where all others have one
    h, args = tl.make(g, M, N, K, R, n, of, N % 16 == 0)
    room = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = room[:M * N].view(M, N)
    size = bq.linear_lora_i8_workspace_bytes(M, N, K, R)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    bq.moe_linear_lora_i8(**args, out=out, ws=ws[:size])
    plain = torch.empty_like(out)
    bq.moe_linear_i8(args["a"], args["a_scale"], args["w"], plain)
    tl.sync()
    rows = np.unique(np.concatenate([[0, 1, M // 2, M - 2, M - 1], g.integers(0, M, 24)]))
    check_rows(out, h, rows, what)
    none = tl.dev(h["of"], torch.int64) < 0
    assert torch.equal(out[none], plain[none])
    assert (room[M * N:] == 7).all() and (ws[size:] == 0xFF).all()


# rows and columns of the tile (weights in rows where N is odd), one or some rows past whole tiles
@pytest.mark.parametrize("tile,M,N", [
    ("32 x 64", 33, 3850), ("64 x 64", 65, 6400), ("64 x 64", 80, 6397), ("128 x 64", 129, 6400), ("128 x 64", 130, 6397),
    ("128 x 128", 129, 16384), ("128 x 128", 150, 16381), ("256 x 128", 257, 15360), ("256 x 128", 290, 15357),
    ("256 x 256", 257, 25600), ("256 x 256", 300, 25597)])
@pytest.mark.parametrize("K", [512, 1088])
@pytest.mark.parametrize("R,n,kind", [(16, 4, "runs"), (72, 9, "rows")])
def test_tiles_with_many_steps_and_rows_past_them(tile, M, N, K, R, n, kind):
    require_gpu()
    run_case(M, N, K, R, n, kind, f"lora tile {tile} M={M} N={N} K={K} R={R} n={n} {kind}")


# enough of A for rows of mixed adapters to be put in order; one and two steps of 16 ranks
@pytest.mark.parametrize("tile,N", [
    ("128 x 64", 1008), ("128 x 64", 1001), ("128 x 128", 3504), ("128 x 128", 3501), ("256 x 128", 4000), ("256 x 128", 4001),
    ("256 x 256", 7296), ("256 x 256", 7301)])
@pytest.mark.parametrize("R,K,kind", [(8, 8192, "rows"), (16, 4096, "rows"), (24, 2752, "rows"), (32, 2112, "runs")])
def test_tiles_of_rows_in_order(tile, N, R, K, kind):
    require_gpu()
    run_case(1100, N, K, R, 24, kind, f"lora in order, tile {tile} N={N} K={K} R={R} {kind}")
