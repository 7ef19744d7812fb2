"""Sizes that reach the kernels of the expert products, each with the plan that it is there for.

tests/test_experts_plan.py asserts the plans on the CPU and tests/test_gpu_expert_variants.py the values
on the GPU, so that a rule that is changed later cannot leave a kernel without a test unnoticed.
"""

# 256 x 256 tiles of a product over rows and their 128 x 128 pieces.
# dtype, out, rows of each expert, rows of no expert, N, K, pad, skew (elements off the allocation)
TILE256 = [
    # a whole round of 256 tiles, then a part-filled one in pieces; last tile rows of 1..128 and of more
    ("bf16", "bf16", [2108, 0, 1992, 1, 2304, 300, 128, 129, 900], 0, 2304, 1024, 0, 0),
    ("bf16", "f32", [2108, 0, 1992, 1, 2304, 300, 128, 129, 900], 70, 2307, 1055, 1, 1),
    ("f16", "f16", [3000, 77, 0, 4500], 0, 2568, 1040, 0, 0),
    ("f16", "f32", [0, 3130, 3999, 641], 5, 2306, 1031, 0, 1),
    # a part-filled round of more than 128 tiles: none in pieces
    ("bf16", "bf16", [1700, 2060], 3, 2312, 1056, 8, 0),
    # every tile in pieces; one expert
    ("f16", "f16", [100, 4000, 90, 60], 0, 2050, 1027, 0, 0),
    ("bf16", "f32", [4001], 0, 2048, 1088, 0, 0),
    # more groups than the lanes of a wave
    ("bf16", "bf16", [17 * (g % 9) for g in range(90)], 0, 1800, 1025, 0, 0),
    # fp32
    ("f32", "f32", [2108, 0, 1992, 1, 2304, 330], 1, 7950, 1024, 0, 0),
    ("f32", "f32", [3001, 4100], 0, 7939, 1029, 1, 1),
    # operands and result past the caches
    ("bf16", "f32", [3000, 1100, 4100], 0, 8200, 1055, 0, 0),
    ("bf16", "bf16", [7000, 5600, 3800], 0, 8192, 1024, 0, 0),
]

# 256 x 256 tiles of the weights' gradient: dtype, out, rows of each expert, rows of no expert, M, N, pad, skew
WGRAD256 = [
    ("bf16", "bf16", [3100, 0, 1005, 1], 0, 2040, 2048, 0, 0),
    ("bf16", "f32", [1, 2111, 1005], 9, 2303, 2090, 1, 1),
    ("f16", "f16", [4093], 0, 3650, 3588, 0, 0),
    ("f16", "f32", [600, 1500, 1024], 0, 2055, 2301, 0, 1),
    ("bf16", "bf16", [2100 * (g % 2) + g % 3 for g in range(121)], 0, 490, 500, 0, 0),     # more than 64 experts
    ("bf16", "bf16", [2000, 900, 0, 1300], 0, 5888, 5800, 0, 0),                           # past the caches
    ("f32", "f32", [1030], 0, 7960, 8190, 0, 0),
    ("f32", "f32", [1025, 1100, 1030, 999], 2, 4093, 4091, 1, 1),                          # past the caches
]

# streamed weights, eight waves: dtype, experts, rows, spare, active, N, K, pad, skew, transposed
STREAM8 = [
    ("bf16", 4, 25, 1, 3, 264, 512, 0, 0, 0), ("bf16", 4, 25, 0, 3, 260, 520, 0, 0, 0),
    ("f16", 3, 20, 0, 3, 135, 531, 1, 1, 0), ("f32", 3, 24, 2, 2, 200, 520, 0, 0, 0), ("f32", 2, 70, 0, 2, 131, 519, 1, 1, 0),
    ("bf16", 4, 25, 1, 3, 72, 2048, 0, 0, 1), ("f16", 4, 25, 0, 3, 45, 2056, 0, 0, 1), ("bf16", 3, 40, 0, 2, 33, 2051, 1, 1, 1),
    ("f32", 3, 24, 2, 2, 70, 1024, 0, 0, 1), ("f32", 2, 30, 0, 2, 41, 1003, 1, 0, 1),
]

# 4-bit products by tile: (tile_m, tile_n), experts, rows, spare, active, N, K, pad
Q4_TILES = [
    ((16, 32), 8, 50, 3, 5, 1035, 300, 1),      # 65 tiles of 16 columns: the last workgroup's second is past them
    ((16, 32), 1, 16, 0, 1, 8193, 640, 0),
    ((16, 32), 4, 160, 5, 3, 1100, 300, 0),     # by the number of rows
    ((16, 32), 1, 200, 0, 1, 1037, 1290, 3),
    ((16, 16), 8, 200, 0, 3, 520, 300, 0),
    ((16, 16), 1, 31, 0, 1, 4100, 390, 2),
]
