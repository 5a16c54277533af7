"""Sizes that reach every tile kernel of the dense operators, with the tile and split chosen for each.  All are
ragged: no size is a multiple of the tiles' rows, columns or slices.  test_dense_plan_cpu.py holds the choice
to this table, test_gpu_dense_tiles.py checks the results."""

# (type, T, K, N, tile rows, contraction split)
LINEAR = [("bf16", 361, 112, 832, 64, False), ("bf16", 141, 1384, 440, 64, True), ("bf16", 3479, 360, 6136, 128, False),
          ("bf16", 943, 4016, 2448, 128, True), ("bf16", 4267, 2016, 3064, 256, False), ("bf16", 2829, 6040, 1448, 256, True),
          ("f32", 77, 216, 2144, 32, False), ("f32", 157, 408, 728, 32, True), ("f32", 2163, 232, 592, 64, False),
          ("f32", 41, 3424, 3800, 64, True), ("f32", 2453, 96, 2472, 128, False), ("f32", 1355, 4752, 352, 128, True)]
# (type, T, H, I, tile rows, contraction split)
GATED = [("bf16", 677, 440, 104, 64, False), ("bf16", 111, 976, 600, 64, True), ("bf16", 2421, 1352, 1312, 128, False),
         ("bf16", 2283, 4176, 528, 128, True), ("bf16", 1571, 1736, 4560, 256, False), ("bf16", 1749, 6192, 1184, 256, True),
         ("f32", 107, 184, 568, 32, False), ("f32", 63, 440, 664, 32, True), ("f32", 2845, 456, 200, 64, False),
         ("f32", 825, 936, 304, 64, True), ("f32", 1359, 112, 2800, 128, False), ("f32", 3361, 1416, 264, 128, True)]
# (type, T, columns of x, columns of dz, tile rows of dx and of dw, split of dx's and of dw's contraction)
GRADIENTS = [("bf16", 159, 272, 336, 64, 128, False, False), ("bf16", 1147, 424, 528, 64, 128, False, True),
             ("bf16", 39, 744, 1600, 64, 128, True, False), ("bf16", 913, 136, 1168, 64, 128, True, True),
             ("bf16", 291, 944, 240, 128, 128, False, False), ("bf16", 1311, 544, 368, 128, 128, False, True),
             ("bf16", 837, 336, 3056, 128, 128, True, False), ("bf16", 875, 432, 1744, 128, 128, True, True),
             ("bf16", 8187, 4104, 4112, 256, 256, False, False),
             ("f32", 73, 496, 544, 32, 128, False, False), ("f32", 1213, 240, 400, 32, 128, False, True),
             ("f32", 107, 112, 2320, 32, 128, True, False), ("f32", 227, 296, 1312, 32, 128, True, True),
             ("f32", 81, 352, 160, 64, 128, False, False), ("f32", 551, 2088, 160, 64, 128, False, True),
             ("f32", 57, 1304, 2480, 64, 128, True, False), ("f32", 353, 600, 976, 64, 128, True, True),
             ("f32", 107, 840, 48, 128, 128, False, False), ("f32", 791, 464, 112, 128, 128, False, True)]
# 256-row tiles whose last round runs as halves: (T, K, N, gated)
HALVES = [(7700, 2056, 7168, False), (3900, 2056, 7168, True)]
