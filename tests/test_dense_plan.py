"""Which kernel moe_gemm_fp8 takes (csrc/dense_plan.h, compiled for the host): the sizes the GPU tests rely on reach the
kernels they are meant for; no workgroup gets an empty share of K; the workspace is that of the shares; and a workspace
that is missing, short or misaligned is refused."""

import ctypes
import os
import subprocess

import pytest

import dense_shapes
import int4_weights_amd as moe

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "int4_weights_amd", "csrc")
KINDS = ["stream16", "stream32", "stream64", "64x64", "64x128", "128x128", "128x128two", "256x256"]
WORKSPACE = 6
P = 1 << 20  # a fake, aligned address: never dereferenced on these paths

SRC = """
#include <stdio.h>
#include "dense_plan.h"
int main() {
  int M, N, K, wide;
  while (scanf("%d %d %d %d", &M, &N, &K, &wide) == 4) {
    const moe::Plan p = moe::plan_dense(M, N, K, wide != 0);
    printf("%d %d %d\\n", (int)p.kind, p.splits, moe::split_blocks(K / 128, p.splits));
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SRC)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-o", str(d / "plan"), str(d / "plan.cpp")], check=True)

    def ask(shapes):
        text = "".join(f"{M} {N} {K} {int(w)}\n" for M, N, K, w in shapes)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return ask


def test_sizes_reach_the_kernels_they_are_meant_for(plan):
    got = plan([s[:4] for s in dense_shapes.ALL])
    for s, (kind, splits, _) in zip(dense_shapes.ALL, got):
        assert (KINDS[kind], splits) == s[4:], s
    for f32 in (False, True):
        reached = {s[4] for s in dense_shapes.ALL if s[3] == f32}
        assert reached == set(KINDS) - {"256x256" if f32 else "128x128two"}


def _grid():
    for M in (65, 66, 100, 131, 200, 257, 300, 451, 1000, 2100):
        for N in (1, 60, 96, 209, 256, 500, 1000, 1100, 2200, 4100):
            for KB in (*range(1, 70), 91, 128, 200, 256):
                yield M, N, 128 * KB


def test_no_share_of_k_is_empty(plan):
    split = 0
    for wide in (False, True):
        shapes = [(*s, wide) for s in _grid()]
        for (M, N, K, _), (_, splits, per) in zip(shapes, plan(shapes)):
            KB = K // 128
            if splits == 1:
                continue
            split += 1
            assert (splits - 1) * per < KB <= splits * per, (M, N, K, wide, splits, per)
            assert per >= 8, "every share but the last has at least 8 blocks"
    assert split > 500


def test_workspace_is_that_of_the_shares(plan):
    shapes = list(_grid())
    n, w = (plan([(*s, wide) for s in shapes]) for wide in (False, True))
    for (M, N, K), a, b in zip(shapes, n, w):
        s = max(a[1], b[1])
        assert moe.moe_gemm_fp8_workspace_bytes(M, N, K) == (4 * s * M * ((N + 3) & ~3) if s > 1 else 0)


@pytest.mark.parametrize("M,N,K", sorted({s[:3] for s in dense_shapes.SPLIT}))
def test_missing_short_and_misaligned_workspaces_are_refused(M, N, K):
    lib = moe.load()
    need = moe.moe_gemm_fp8_workspace_bytes(M, N, K)
    assert need > 0
    for ws, size in ((None, need), (P, need - 1), (P, 0), (P + 8, need)):
        for out in (0, 1):
            assert lib.moe_gemm_fp8(ctypes.c_void_p(P), K, ctypes.c_void_p(P), ctypes.c_void_p(P), K, ctypes.c_void_p(P), 128,
                                    ctypes.c_void_p(P), out, N, None, 0, M, N, K, ctypes.c_void_p(ws), size,
                                    None) == WORKSPACE
