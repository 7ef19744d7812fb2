"""Sizes that reach the kernels of a feed-forward block's operators, each with the plan that it is there
for: tests/test_ffn_plan.py asserts the plans on the CPU, tests/test_gpu_ffn_variants.py the values on
the GPU.
"""

UNEVEN = [2108, 0, 1992, 1, 2304, 300, 128, 129, 900]

# plan, dtype, rows of each expert, rows of none, N, K, pad, skew, transposed
GATED = [
    (dict(tile_m=256, tile_n=128, pieces=1, pipeline=1), "bf16", UNEVEN, 70, 1152, 1024, 0, 0, 0),
    (dict(tile_m=256, tile_n=128, pieces=1, pipeline=1), "f16", UNEVEN, 0, 1147, 1055, 1, 1, 0),
    (dict(tile_m=256, tile_n=128, pieces=1, pipeline=1), "bf16", [4001, 4160], 3, 1096, 1048, 8, 0, 1),
    (dict(tile_m=256, tile_n=128, pieces=1, pipeline=1), "f16", [100, 4000, 4090, 60], 0, 1051, 1027, 0, 1, 1),
    (dict(tile_m=128, tile_n=64, pieces=0, pipeline=0), "bf16", UNEVEN, 5, 600, 264, 0, 0, 0),
    (dict(tile_m=128, tile_n=64, pieces=0, pipeline=0), "f16", [8000], 0, 515, 131, 1, 1, 1),
    (dict(tile_m=128, tile_n=64, pieces=0, pipeline=0), "bf16", [1300], 0, 1032, 2056, 1, 0, 0),
    (dict(tile_m=64, tile_n=64, splits=2), "bf16", [450, 1, 0, 261], 9, 400, 2088, 1, 0, 1),
    (dict(tile_m=64, tile_n=64, splits=2), "f16", [257], 0, 1001, 4101, 0, 1, 0),
    (dict(tile_m=64, tile_n=64, splits=8, pipeline=0), "f32", [325], 0, 104, 2050, 0, 0, 1),
    (dict(tile_m=64, tile_n=64, splits=1), "bf16", [300, 77, 0, 900], 9, 200, 520, 0, 0, 1),
    (dict(tile_m=64, tile_n=64, splits=4), "f16", [100], 0, 1030, 1050, 0, 0, 0),
    (dict(tile_m=64, tile_n=64, splits=2), "bf16", [30, 41, 0, 7], 3, 264, 600, 1, 0, 1),
    (dict(tile_m=64, tile_n=64, splits=4, pipeline=0), "f32", [50], 0, 333, 700, 0, 1, 0),
    (dict(tile_m=64, tile_n=64, pipeline=1), "f32", [700, 0, 333], 4, 300, 129, 1, 0, 1),
    (dict(kernel="stream", waves=8, splits=4), "bf16", [5], 0, 100, 4100, 1, 0, 1),
    (dict(kernel="stream", waves=8, splits=4), "f32", [16], 0, 130, 1100, 0, 0, 0),
]

# plan, dtype, rows of each expert, rows of none, N, K, pad, skew, transposed
GRAD = [
    (dict(tile_m=256, tile_n=256, pieces=1, pipeline=1), "bf16", UNEVEN, 70, 1152, 1024, 0, 0, 1),
    (dict(tile_m=256, tile_n=256, pieces=1, pipeline=1), "f16", UNEVEN, 0, 1147, 1055, 1, 1, 0),
    (dict(tile_m=256, tile_n=256, pieces=1, pipeline=1), "bf16", [4001, 4160], 3, 1096, 1048, 8, 0, 0),
    (dict(tile_m=256, tile_n=256, pieces=1, pipeline=1), "f32", [2108, 0, 1992, 1, 2304, 330], 1, 7950, 1024, 0, 0, 1),
    (dict(tile_m=64, tile_n=128), "bf16", UNEVEN, 5, 600, 264, 0, 0, 1),
    (dict(tile_m=64, tile_n=128), "f16", [8000], 0, 515, 131, 1, 1, 0),
    (dict(tile_m=64, tile_n=64, pipeline=0), "bf16", [300, 77, 0, 900], 9, 200, 520, 0, 0, 0),
    (dict(tile_m=64, tile_n=128, pipeline=0), "f16", [700], 0, 4100, 2050, 0, 1, 1),
    (dict(tile_m=64, tile_n=64, pipeline=1), "f32", [700, 0, 333], 4, 300, 129, 1, 0, 1),
    (dict(kernel="stream"), "bf16", [5, 0, 9], 1, 100, 410, 1, 0, 1),
]

# plan, dtype, adapters with rows, rows, rows of none, N, K, rank, pad, skew, transposed
ADAPTERS = [
    (dict(tile_m=256, pieces=1, pipeline=1), "bf16", 5, 4100, 100, 2060, 1024, 40, 0, 0, 0),
    (dict(tile_m=256, pieces=1, pipeline=1), "f16", 70, 4230, 0, 2059, 1031, 16, 1, 1, 1),
    (dict(tile_m=256, pieces=1, pipeline=1), "bf16", 1, 4096, 0, 2048, 1056, 100, 0, 0, 1),
    (dict(tile_m=256, splits=2, pieces=0, pipeline=1), "bf16", 5, 2100, 100, 2060, 6200, 40, 0, 0, 0),
    (dict(tile_m=256, splits=2, pieces=0, pipeline=1), "f16", 70, 1807, 0, 2307, 6231, 16, 1, 1, 1),
    (dict(tile_m=128, splits=1), "f16", 9, 4100, 33, 1100, 264, 8, 0, 0, 0),
    (dict(tile_m=128, splits=1), "bf16", 3, 5000, 0, 1001, 131, 33, 1, 1, 1),
    (dict(tile_m=64, splits=4), "bf16", 7, 300, 20, 520, 1100, 24, 0, 0, 1),
    (dict(tile_m=64, splits=8), "f16", 150, 260, 0, 300, 2050, 7, 1, 0, 0),
    (dict(tile_m=64, splits=1), "f16", 30, 512, 9, 1536, 520, 17, 0, 1, 1),
    (dict(tile_m=128, splits=4), "bf16", 7, 1025, 20, 520, 2100, 24, 0, 0, 1),
    (dict(tile_m=128, splits=8), "f16", 150, 1060, 0, 300, 4106, 7, 1, 0, 0),
    (dict(tile_m=64, splits=1, pipeline=1), "f32", 41, 1333, 21, 771, 201, 5, 0, 0, 0),
    (dict(tile_m=64, splits=4, pipeline=0), "f32", 6, 300, 3, 264, 520, 20, 1, 1, 1),
    (dict(tile_m=64, splits=4, pipeline=1), "f32", 6, 1300, 3, 264, 1030, 20, 1, 1, 1),
    (dict(kernel="tiles", tile_m=64, splits=4), "bf16", 20, 64, 7, 512, 1024, 32, 0, 0, 1),
    (dict(kernel="tiles", tile_m=64, splits=4), "f32", 5, 40, 0, 300, 520, 9, 1, 0, 0),
    (dict(kernel="stream", splits=8), "bf16", 3, 7, 1, 300, 4104, 16, 0, 0, 1),
    (dict(kernel="stream", splits=8), "f32", 2, 16, 0, 130, 1100, 300, 0, 0, 0),
    (dict(kernel="stream"), "f16", 2, 3000, 5, 7, 200, 8, 0, 0, 0),
]
