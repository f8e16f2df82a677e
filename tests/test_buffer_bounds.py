"""Where loads through buffers lie (CPU).  A buffer's bound holds for a load's vector offset alone,
so a load that may pass the end says so there; and the adapters' first product of a tile that
passes the last row is read inside its own bytes or as zeros."""
import os
import re
import shutil
import subprocess

import pytest

import bit_quantized_grouped_amd as bq
from bit_quantized_grouped_amd import build as bqb

PAST = ("past", "voff_oob", "kPast", "0xFFFFFFF0u")   # marks of an offset past every buffer


def calls(text, name):
    """Argument lists of the calls of `name`."""
    for m in re.finditer(rf"\b{name}\(", text):
        depth, args, at = 1, [""], m.end()
        while depth:
            c = text[at]
            depth += (c in "([{") - (c in ")]}")
            if c == "," and depth == 1:
                args.append("")
            elif depth:
                args[-1] += c
            at += 1
        yield [" ".join(a.split()) for a in args]


@pytest.mark.parametrize("source", [s for s in bqb.SOURCES if s != "gemm_q4.hip"])
def test_no_bound_hangs_on_a_scalar_offset(source):
    """A scalar offset is 0, or the vector offset can carry a mark of its own."""
    text = open(os.path.join(bqb.CSRC, source)).read()
    for name in ("buf_to_lds16", "buf_load16_u"):
        for args in calls(text, name):
            voff, soff = args[-2], args[-1]
            assert soff == "0" or any(p in voff for p in PAST), f"{source}: {name}({', '.join(args)})"


TABLE = r"""
#include "moe_lora.h"
#include <cstdio>
#include <cstdlib>
using namespace moeq4;
int main(int argc, char** argv) {
    const int M = atoi(argv[1]), rank = atoi(argv[2]), steps = (rank + 15) / 16;
    const size_t all = lora_u_bytes(((size_t)M + 15) / 16, steps);
    for (int rows : {32, 64, 128, 256}) {
        size_t last = 0, zeros = 0;
        for (int m0 = 0; m0 < M; m0 += rows) {
            const int in = rows / 16 < (M - m0 + 15) / 16 ? rows / 16 : (M - m0 + 15) / 16;
            const size_t base = lora_u_at(m0 / 16, 0, steps, 0), bytes = lora_u_bytes(in, steps);
            for (int t = 0; t < rows / 16; ++t)
                for (int s = 0; s < steps; ++s)
                    for (int lane = 0; lane < 64; ++lane) {
                        const size_t at = (uint32_t)lora_u_at(t, s, steps, lane);
                        if (at < bytes) last = base + at + 16 > last ? base + at + 16 : last;
                        else ++zeros;
                    }
        }
        printf("%d %zu %zu %zu\n", rows, last, all, zeros);
    }
}
"""


@pytest.fixture(scope="module")
def table(tmp_path_factory):
    if not shutil.which(bqb.hipcc()):
        pytest.skip("no hipcc")
    d = tmp_path_factory.mktemp("u")
    (d / "u.hip").write_text(TABLE)
    cmd = [bqb.hipcc(), "--offload-host-only", "-std=c++17", "-O1", "-I", os.path.join(bqb.ROOT, "include"), "-I", bqb.CSRC,
           str(d / "u.hip"), "-o", str(d / "u")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return str(d / "u")


@pytest.mark.parametrize("M,N,rank", [
    (17, 4096, 8), (130, 8192, 16), (130, 8192, 64), (200, 4096, 128), (300, 28672, 64), (257, 4096, 128), (333, 1001, 8),
    (1023, 48, 40), (8192, 4096, 64), (8193, 4096, 72)])
def test_reads_of_the_first_product_end_with_it(table, M, N, rank):
    """For every height of a tile: the last byte that is read is u's last, and what a tile asks for
    behind the rows' lies past its buffer, where a load gives zeros."""
    out = subprocess.run([table, str(M), str(rank)], capture_output=True, text=True, check=True).stdout
    steps = (rank + 15) // 16
    for line in out.split("\n")[:-1]:
        rows, last, size, zeros = (int(v) for v in line.split())
        assert last == size == (M + 15) // 16 * steps * 1024
        past = -(-M // rows) * rows // 16 - (M + 15) // 16   # 16-row tiles behind the last row's
        assert zeros == past * steps * 64
        assert size <= bq.linear_lora_i8_workspace_bytes(M, N, 1024, rank)
