"""Which kernel moe_gemm_bf16 takes (csrc/linear_plan.h, compiled for the host): the sizes of the GPU tests reach every kernel
they are meant for; no workgroup gets an empty share of K; shares fit the chip; the workspace is that of the shares."""

import os
import random
import subprocess

import pytest

import int4_weights_amd as moe
from linear_shapes import KINDS, REACHED

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "int4_weights_amd", "csrc")
SRC = """
#include <stdio.h>
#include "linear_plan.h"
int main() {
  int M, N, K, tr;
  while (scanf("%d %d %d %d", &M, &N, &K, &tr) == 4) {
    const moe::LinPlan p = moe::plan_linear(M, N, K, tr != 0);
    int bm = 0, bn = 0;
    for (const moe::LinTile& t : moe::kLinTiles)
      if (t.kind == p.kind) bm = t.bm, bn = t.bn;
    printf("%d %d %d %d %d\\n", (int)p.kind, p.splits, moe::lin_split_blocks((K + 63) / 64, p.splits), bm, bn);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SRC)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-o", str(d / "plan"), str(d / "plan.cpp")], check=True)

    def ask(shapes):
        text = "".join(f"{M} {N} {K} {int(t)}\n" for M, N, K, t in shapes)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return ask


def test_sizes_reach_the_kernels_they_are_meant_for(plan):
    for order, want in REACHED.items():
        got = plan([(*s, order != "nt") for s in want])
        assert {s: (KINDS[g[0]], g[1]) for s, g in zip(want, got)} == want
        tiles = set(KINDS) if order == "nt" else {k for k in KINDS if not k.startswith("stream")}
        assert {k for k, _ in want.values()} == tiles
        assert {s for _, s in want.values()} - {1}  # some in shares


def test_shares_and_workspace(plan):
    r = random.Random(5)
    sizes = [(r.choice([1, 7, 64, 65, 200, 900, 5000]) * r.randint(1, 4), 8 * r.randint(1, 700), 8 * r.choice([1, 9, 100, 900, 5000]))
             for _ in range(600)]
    a, b = plan([(*s, False) for s in sizes]), plan([(*s, True) for s in sizes])
    assert any(p[1] > 1 for p in a) and any(p[1] > 1 for p in b)
    for (M, N, K), p, q in zip(sizes, a, b):
        KB = (K + 63) // 64
        for kind, splits, per, bm, bn in (p, q):
            assert 1 <= splits <= 8 and per * (splits - 1) < KB <= per * splits
            if splits > 1:
                assert per >= 4 and -(-M // bm) * -(-N // bn) * splits <= 256
        assert q[0] >= KINDS.index("64x64") and (M <= 64 or p[0] >= KINDS.index("64x64"))
        need = max(p[1], q[1])
        got = moe.moe_gemm_bf16_workspace_bytes(M, N, K)
        # each share holds M rows of N columns, those of a gated product in two halves of whole vectors
        assert got == 0 if need == 1 else need * M * (2 * (-(-(N // 2) // 4) * 4)) * 4 <= got <= need * M * (N + 8) * 4


def test_no_products_and_no_rows(plan):
    assert [p[1] for p in plan([(5, 8, 0, False), (500, 800, 0, True), (0, 8, 64, False)])] == [1, 1, 1]
