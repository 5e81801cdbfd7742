"""Sizes that reach every kernel of the FP8 linear layer and both forms of the
cross attention on 148 SMs: the plan's choice is checked on the CPU, the
results on a GPU."""

# M, N, K, kernel (0: the one for few rows, else the tile width), its K slices
PRODUCTS = [
    # up to 16 tokens
    (16, 40000, 272, 0, 1), (2, 9480, 400, 0, 2), (9, 5000, 1552, 0, 4), (3, 328, 11648, 0, 8),
    # up to 32
    (32, 19008, 272, 0, 1), (20, 9224, 1040, 0, 2), (24, 4104, 528, 0, 4), (17, 264, 1040, 0, 8),
    # up to 64
    (40, 18952, 528, 0, 1), (34, 9224, 8208, 0, 2), (40, 4616, 4112, 0, 4), (33, 264, 4112, 0, 8),
    (64, 512, 8192, 0, 8),
    # up to 128
    (65, 37904, 144, 0, 1), (65, 7176, 4112, 0, 2), (77, 12688, 3680, 0, 2), (127, 5000, 6160, 0, 4),
    (128, 4616, 8208, 0, 4), (94, 328, 11648, 0, 8), (100, 1032, 4112, 0, 8), (127, 264, 8208, 0, 8),
    # more, or where the weight's tiles would be too few
    (128, 320, 512, 64, 4), (300, 520, 528, 64, 4), (600, 2056, 272, 128, 2), (700, 4616, 1040, 256, 4),
]

# batch, sequences of keys, queries, keys, heads, key/value heads, head size, split form?
ATTENTION = [
    (3, 1, 520, 390, 60, 30, 64, False), (3, 1, 520, 390, 60, 30, 120, False), (5, 1, 300, 200, 60, 20, 128, False),
    (3, 1, 1, 1500, 8, 2, 128, True), (3, 1, 40, 700, 4, 4, 64, True),
]
