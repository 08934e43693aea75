"""Sizes of moe_gemm_fp8 with long K for each of its kernels: (M, N, K, fp32 output, kernel, workgroups that share K).

K blocks (K / 128): 13 and 59 leave a group of 4 scales unfinished, 16 and 56 do not; 41 and 52 share badly.  Every ring
of slots is refilled several times and the scales' buffers are used again.
"""

STREAM = [(M, N, K, f32, kind, 1) for M, kind in ((9, "stream16"), (30, "stream32"), (60, "stream64"))
          for N in (300, 4200) for K in (7168, 7552) for f32 in (False, True)]
STREAM += [(500, 500, 6656, f32, "stream64", 1) for f32 in (False, True)]

TILES = []
for _K in (1664, 2048, 7168):
    TILES += [(131, 7168, _K, False, "64x128", 1), (131, 7168, _K, True, "64x128", 1),
              (1100, 3000, _K, False, "128x128", 1), (1100, 3000, _K, True, "128x128", 1),
              (1030, 4100, _K, True, "128x128two", 1), (2100, 4500, _K, False, "256x256", 1)]
TILES += [(300, 1100, K, f32, "64x64", 1) for K in (1664, 2048) for f32 in (False, True)]

# K shared by several workgroups
SPLIT = [(100, 96, 7168, f32, "64x64", 7) for f32 in (False, True)]
SPLIT += [(100, 96, 7552, f32, "64x64", 5) for f32 in (False, True)]
SPLIT += [(131, 256, 7168, f32, "64x64", 7) for f32 in (False, True)]
SPLIT += [(131, 2200, K, f32, "64x64", 2) for K in (5248, 7168) for f32 in (False, True)]
SPLIT += [(66, 60, 6656, True, "64x64", 5), (131, 256, 6656, True, "64x64", 5)]

ALL = STREAM + TILES + SPLIT
