"""Sizes (bits of x, tokens, sum, columns of y) of the product on 4-bit weights
that take each of its kernels in turn, shared by the check of that (CPU) and
the products themselves (GPU): ragged in all three directions, short sums
and, on 8-bit rows, sums behind the blocks whose exponents a workgroup holds."""

PRODUCTS = [
    # few tokens
    (4, 7, 1352, 1000), (4, 16, 9736, 264), (8, 7, 1352, 1000), (8, 13, 9736, 264),
    (4, 650, 440, 11448), (8, 650, 440, 11448), (8, 1795, 3744, 5456),      # 256 x 256
    (4, 258, 440, 14664), (8, 258, 440, 14664), (8, 297, 3640, 14072),      # 256 x 128
    (4, 257, 616, 11344), (8, 257, 616, 11344), (8, 257, 3960, 11704),      # 128 x 160
    (4, 138, 392, 11240), (8, 138, 392, 11240), (8, 130, 3616, 14824),      # 128 x 128
    (4, 141, 912, 12216), (8, 144, 1304, 11440), (8, 137, 3864, 11896),     # 128 x 96
    (4, 65, 520, 6760), (8, 4370, 528, 72), (8, 66, 3912, 13384),           # 64 x 64
    (4, 98, 920, 4232), (8, 65, 1784, 8528), (8, 69, 8136, 8616),           # 64 x 96, the sum in two parts
    (4, 65, 1888, 6040), (8, 4316, 1784, 80), (8, 4663, 14456, 72),         # 64 x 64, in four
    (4, 35, 1584, 4136), (8, 35, 1584, 4136), (8, 36, 14504, 4168),         # 32 x 64, in four
    (4, 35, 2168, 40), (8, 35, 2168, 40), (8, 33, 14440, 40),               # 32 x 32, in four
]

# Sums so long that a workgroup fetches the exponents of 8-bit rows three times, for every tile.
LONG_SUMS = [
    (8, 1795, 7400, 5456),      # 256 x 256
    (8, 385, 7400, 11016),      # 256 x 128
    (8, 257, 7400, 11704),      # 128 x 160
    (8, 130, 7400, 14824),      # 128 x 128
    (8, 137, 7400, 11896),      # 128 x 96
    (8, 66, 7400, 13384),       # 64 x 64
    (8, 65, 15000, 8528),       # 64 x 96, the sum in two parts
    (8, 65, 29000, 6040),       # 64 x 64, in four
    (8, 36, 29000, 4168),       # 32 x 64, in four
    (8, 33, 29000, 40),         # 32 x 32, in four
]
