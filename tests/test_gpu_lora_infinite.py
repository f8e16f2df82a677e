"""Infinities and NaN in adapters: moe_linear_lora_i8 gives what its definition does, element by
element, in every form of the product.  Tolerances of finite values as in test_gpu_lora."""
import numpy as np
import pytest
import torch

import bit_quantized_grouped_amd as bq
import test_gpu_lora as tl
from gpu_cases import DEV, announce, require_gpu
from oracle import serve_oracle

pytestmark = pytest.mark.gpu

# a size of each form: 16 x 16, 16 x 32, 32 x 32 and 32 x 64 with K over waves, then the tiles
# through LDS from 32 x 64 to 256 x 256; the last two with rows in order of their adapters
FORMS = [(6, 64, 192), (15, 160, 1024), (17, 4096, 128), (64, 4096, 128), (128, 4096, 192), (33, 3850, 512), (80, 6397, 256),
         (129, 6400, 128), (129, 16384, 128), (290, 15357, 128), (257, 25600, 128), (1100, 1008, 4096), (1100, 4001, 4096)]


def case(M, N, K):
    g = np.random.default_rng(M + N)
    n = 24 if K == 4096 else 6
    of = tl.pattern(g, M, n, "rows")
    of[:6] = [0, 1, 2, 3, -1, 1]
    h, args = tl.make(g, M, N, K, 16, n, of, N % 16 == 0)
    h["a"][h["a"] == 0] = 1   # 0 times an infinity is NaN in the definition too
    args["a"].copy_(torch.from_numpy(h["a"]))
    return h, args


def compare(out, clean, h, touched, what):
    """Rows of the touched adapters against the definition; all others as they were, bit for bit."""
    of = h["of"]
    keep = tl.dev(~np.isin(of, touched), torch.bool)
    assert torch.equal(out[keep], clean[keep]), what
    rows = np.unique(np.concatenate([np.nonzero(of == j)[0][:3] for j in touched]))
    with np.errstate(invalid="ignore"):
        want, size = serve_oracle.linear_lora(h["a"][rows], h["sa"][rows], h["w"], h["sw"], h["A"], h["B"], h["s"], of[rows])
        K, R = h["a"].shape[1], h["A"].shape[1]
        off = size * (2.0 ** -16 + (K + 2 * R + 16) * 2.0 ** -24) + 8 * 2.0 ** -24 * (np.abs(want) + size)
        bound = tl.HALF * (np.abs(want) + off) + off
        got = out[torch.from_numpy(rows).to(DEV)].double().cpu().numpy()
        err = np.abs(got - want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN"
    assert np.array_equal(np.isinf(got), np.isinf(want)) and (got[np.isinf(want)] == want[np.isinf(want)]).all(), f"{what}: inf"
    at = np.isfinite(want)
    assert (err[at] <= bound[at]).all(), f"{what}: finite values"
    return want


def run(h, args, put, touched, what):
    M, N = len(h["a"]), len(h["w"])
    announce(what)
    ws = tl.workspace(M, N, h["a"].shape[1], 16)
    clean, out = (torch.empty((M, N), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    bq.moe_linear_lora_i8(**args, out=clean, ws=ws)
    for name, at, value in put:
        h[name][at] = value
        getattr(args["adapters"], name.lower())[at] = value
    bq.moe_linear_lora_i8(**args, out=out, ws=ws)
    tl.sync()
    return compare(out, clean, h, touched, what)


@pytest.mark.parametrize("M,N,K", FORMS)
def test_infinities_in_the_first_matrix(M, N, K):
    """The adapter's u is infinite for a rank: infinities of B's signs, NaN where B is 0."""
    require_gpu()
    h, args = case(M, N, K)
    put = [("A", (1, 3, 7), np.inf), ("B", (1, 0, 3), 0.0), ("A", (2, 0, K - 1), -np.inf), ("A", (3, 5, 9), np.nan)]
    want = run(h, args, put, [1, 2, 3], f"lora, infinity in A, M={M} N={N} K={K}")
    assert np.isinf(want).any() and not np.isfinite(want).any()


@pytest.mark.parametrize("M,N,K", FORMS)
def test_infinities_in_the_second_matrix(M, N, K):
    """They reach their column of their adapter's rows, and nothing else."""
    require_gpu()
    h, args = case(M, N, K)
    put = [("B", (1, 0, 5), np.inf), ("B", (1, N // 2, 15), -np.inf), ("B", (2, N - 1, 0), -np.inf), ("B", (3, 7, 8), np.nan),
           ("B", (3, 8, 2), np.inf), ("B", (3, 8, 3), np.inf)]
    want = run(h, args, put, [1, 2, 3], f"lora, infinity in B, M={M} N={N} K={K}")
    assert np.isinf(want).any() and np.isnan(want).any() and np.isfinite(want).mean() > 0.9


@pytest.mark.parametrize("M,N,K", FORMS)
def test_infinities_that_meet(M, N, K):
    """An infinite u at the rank of an infinite b, and two infinite ranks in one column."""
    require_gpu()
    h, args = case(M, N, K)
    put = [("A", (1, 3, 7), np.inf), ("B", (1, 2, 3), -np.inf), ("A", (2, 15, 1), -np.inf), ("A", (2, 0, 2), np.inf),
           ("B", (2, N - 1, 15), np.inf), ("B", (0, 5, 0), np.inf), ("B", (0, 5, 9), -np.inf)]
    want = run(h, args, put, [0, 1, 2], f"lora, infinities that meet, M={M} N={N} K={K}")
    assert np.isinf(want).any() and np.isnan(want).any() and np.isfinite(want).any()
