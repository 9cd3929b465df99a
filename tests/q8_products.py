"""Sizes (tokens, sum, columns of y) of the 8-bit product that take each of its
kernels in turn, shared by the check of that (CPU) and the products themselves
(GPU): every size ragged in all three directions, short sums and sums behind
the blocks whose exponents a workgroup holds at a time."""

PRODUCTS = [
    (7, 1352, 1000), (16, 9736, 264),                            # few tokens
    (1158, 1160, 8416), (1675, 7744, 8688),                      # 256 x 256
    (133, 624, 8648), (158, 592, 8232),                          # 128 x 128, two stages
    (262, 672, 8440), (259, 7776, 8280),                         # 128 x 128, three stages
    (259, 1064, 11784), (257, 7800, 10984),                      # 128 x 160
    (129, 696, 8496), (131, 7824, 8208),                         # 128 x 96
    (164, 568, 2848), (2752, 584, 136), (134, 7760, 3272),       # 128 x 64
    (35, 2056, 4920), (33, 30944, 4216),                         # 32 x 64, the sum in four parts
    (54, 2312, 40), (33, 30960, 48),                             # 32 x 32, the sum in four parts
]
