"""The sizes of the epilogue tests reach the kernels and shares that they are meant for (csrc/linear_plan.h, compiled for the host)."""

import random

from linear_epilogue_shapes import EPILOGUES, SHARES
from linear_shapes import KINDS
from test_linear_plan import plan  # noqa: F401  (a fixture)


def test_sizes_reach_the_kernels_they_are_meant_for(plan):  # noqa: F811
    for transposed, table in ((False, EPILOGUES), (True, SHARES["nn"]), (True, SHARES["tn"])):
        got = plan([(*s, transposed) for s in table])
        assert {s: (KINDS[g[0]], g[1]) for s, g in zip(table, got)} == table


def test_every_kernel_is_reached_whole_and_in_shares(plan):  # noqa: F811
    r = random.Random(3)
    sizes = [(int(2 ** r.uniform(0, 13.5)), 2 * int(2 ** r.uniform(0, 12.5)), 8 * int(2 ** r.uniform(0, 13)), False) for _ in range(20000)]
    some = {(KINDS[g[0]], g[1] > 1) for g in plan(sizes)}
    assert some == {(kind, shares > 1) for kind, shares in EPILOGUES.values()}
