"""How moe_experts_decode divides its work (csrc/decode_plan.h, compiled for the host): no more persistent workgroups than run at once;
everything fits the LDS; the sizes of the GPU tests reach every kernel that any size reaches."""

import os
import random
import subprocess

import pytest

from decode_shapes import COMPUTE_UNITS, FORMATS, REACHED

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "int4_weights_amd", "csrc")
LDS = 160 * 1024
SRC = """
#include <stdio.h>
#include "decode_plan.h"
int main() {
  int f, T, k, E, H, I, cus;
  while (scanf("%d %d %d %d %d %d %d", &f, &T, &k, &E, &H, &I, &cus) == 7) {
    const moe::DecodePlan p = moe::plan_decode(f, T, k, E, H, I, cus);
    printf("%d %d %d %d %d %d %d %d %d\\n", p.rows, p.up_waves, p.up_groups, p.down_waves, p.down_ring, p.ksplit,
           moe::dec_up_lds(f, p.rows, p.up_waves, T * k), moe::dec_down_lds(p.down_waves, p.down_ring, p.ksplit, T * k),
           moe::dec_up_cols(f));
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SRC)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-o", str(d / "plan"), str(d / "plan.cpp")], check=True)

    def ask(calls):
        text = "".join(" ".join(map(str, c)) + "\n" for c in calls)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return ask


def sizes(n, cus):
    r = random.Random(11)
    for _ in range(n):
        k = r.choice([1, 2, 4, 6, 8, 16, 64, r.randint(1, 64)])
        T = min(r.randint(1, 128), 1024 // k, 128 if r.random() < 0.7 else 12)
        yield (r.randrange(4), T, k, int(2 ** r.uniform(0, 10)), 128 * r.choice([1, 8, 32, 33, 56, 256]),
               128 * r.choice([1, 2, 6, 11, 16, 256]), cus)


def on_a_unit(lds):
    return 2 if 2 * lds <= LDS else 1


@pytest.mark.parametrize("cus", [256, 304, 20])
def test_workgroups_run_at_once_and_fit(plan, cus):
    calls = list(sizes(20000, cus))
    for (f, T, k, E, H, I, _), (rows, up_waves, groups, down_waves, ring, ksplit, up, down, cols) in zip(calls, plan(calls)):
        R, blocks = T * k, I // (64 if f == 0 else 128)
        assert rows in (4, 8, 16) and (rows > 4 or f > 0)
        assert up <= LDS and down <= LDS
        assert groups == min(R * (I // cols), on_a_unit(up) * cus)  # persistent: more would begin when others have ended
        assert ksplit == 1 or (ksplit <= blocks and (ksplit // 2) * R < down_waves)


def test_sizes_reach_every_kernel(plan):
    up, down = set(), set()
    calls = list(sizes(40000, COMPUTE_UNITS))
    for c, p in zip(calls, plan(calls)):
        up.add((c[0], p[0], p[1], on_a_unit(p[6])))
        down.add((c[0], p[0], p[3], p[4] // 1024))
    for f, name in enumerate(FORMATS):
        want = REACHED[name]
        got = plan([(f, *s, COMPUTE_UNITS) for s in want])
        assert {s: (p[0], p[1], on_a_unit(p[6]), p[3], p[4] // 1024) for s, p in zip(want, got)} == want
        assert {(v[0], v[1], v[2]) for v in want.values()} == {u[1:] for u in up if u[0] == f}
        assert {(v[0], v[3], v[4]) for v in want.values()} == {d[1:] for d in down if d[0] == f}
