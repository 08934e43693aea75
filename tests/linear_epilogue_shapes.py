"""Sizes of the dense bf16 product's epilogue tests and the kernel and shares of K that each reaches (kinds as in csrc/linear_plan.h):
every tile with whole tiles and with edges, and every tile that is ever split with shares.  N / 2 is no multiple of 4 in most: a
gated product's halves begin at odd places."""

# (M, N, K): (kind, shares of K)
EPILOGUES = {
    (9, 202, 1288): ("stream16", 1),
    (30, 202, 520): ("stream32", 1),
    (45, 202, 520): ("stream64", 1),
    (131, 202, 2056): ("64x64", 1),
    (70, 202, 8200): ("64x64", 5),
    (500, 4096, 200): ("64x128", 1),
    (71, 3430, 8376): ("64x128", 4),
    (1000, 4094, 712): ("128x128", 1),
    (1024, 4096, 96): ("128x128", 1),
    (900, 902, 16392): ("128x128", 4),
    (2050, 2602, 136): ("128x128two", 1),
    (2048, 2560, 136): ("128x128two", 1),
    (2300, 4090, 136): ("256x256", 1),
    (2304, 4096, 136): ("256x256", 1),
    (1035, 1962, 6752): ("256x256", 6),
}
# products in the gradients' orders with shares, of the tiles whose shares linear_shapes does not reach
SHARES = {
    "nn": {(72, 3432, 8376): ("64x128", 4), (1040, 1960, 6752): ("256x256", 6)},
    "tn": {(72, 3432, 8371): ("64x128", 4), (1040, 1960, 6747): ("256x256", 6)},
}
