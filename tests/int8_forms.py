"""Sizes of the 8-bit product for each of the forms that it takes, edges in every operand."""

# form, parts of K, tokens, outputs, K.  256 x 256 tiles: edge rows in both operands, K short of a
# step, odd numbers of steps, a last band of fewer than 8 token tiles (2860 tokens: 12 tiles).
SHAPES = [
    ("few", 1, 3, 16401, 272), ("few", 1, 16, 16384, 1040), ("few", 1, 11, 700, 4000),
    ("32", 1, 17, 1000, 912), ("32", 7, 31, 4103, 7888), ("32", 7, 2, 8200, 8208),
    ("64", 1, 65, 33000, 400), ("64", 3, 120, 5001, 3216), ("64", 1, 500, 8000, 656),
    ("128", 1, 700, 6200, 6160), ("128", 6, 150, 3100, 6160), ("128", 1, 4200, 3900, 400),
    ("256", 1, 1100, 8101, 272), ("256", 1, 2300, 5000, 656), ("256", 1, 3900, 4000, 16), ("256", 1, 3850, 4090, 272), ("256", 1, 2860, 5200, 656),
    ("256", 1, 4095, 3841, 144), ("256", 1, 4090, 4001, 1040),
]
