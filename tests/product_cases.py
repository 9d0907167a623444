"""Cases of the grouped products by the tile that the host's rule gives them:
(product, rows per expert, N, K, (rows, columns) of the tile).

The rule looks at the mean number of rows and at the number of tiles, so a
kernel of large tiles needs a case with many of them.  Each kernel has sums of
an odd and an even number of steps (64 z, FP4 256), ends inside a step's first
and second half, ragged row tiles, more than one column tile with a partial
last one, and experts without rows."""

FORWARD, ROW_GRADIENT, WEIGHT_GRADIENT, FOUR_BITS = 0, 1, 2, 3

CASES = [
    (FORWARD, [16, 0, 33, 1], 200, 328, (64, 128)),
    (FORWARD, [130, 0, 257, 31], 264, 448, (64, 128)),          # few of the larger tiles
    (FORWARD, [523, 0, 900, 177], 2056, 328, (128, 256)),       # 5 steps and 8 of 64 z
    (FORWARD, [523, 0, 900, 177], 2056, 384, (128, 256)),       # 6
    (FORWARD, [1000, 1, 600], 2120, 488, (128, 256)),           # 7 and 40
    (FORWARD, [131] * 13, 2064, 64, (128, 256)),                # 1
    (FORWARD, [2600, 0, 1900], 2056, 328, (256, 256)),
    (FORWARD, [2600, 0, 1900], 2056, 448, (256, 256)),          # 7
    (FORWARD, [4399], 2072, 488, (256, 256)),
    (FORWARD, [4400], 2072, 40, (256, 256)),                    # less than one
    (ROW_GRADIENT, [16, 0, 33, 1], 328, 200, (128, 256)),
    (ROW_GRADIENT, [523, 0, 900, 177], 488, 2056, (128, 256)),
    (ROW_GRADIENT, [523, 0, 900, 177], 448, 2056, (128, 256)),
    (ROW_GRADIENT, [2600, 0, 1900], 328, 2056, (256, 256)),
    (ROW_GRADIENT, [2600, 0, 1900], 384, 2056, (256, 256)),
    (ROW_GRADIENT, [4399], 488, 2072, (256, 256)),
    (ROW_GRADIENT, [4400], 40, 2072, (256, 256)),
    (WEIGHT_GRADIENT, [700, 0, 321], 1032, 1288, (256, 256)),
    (WEIGHT_GRADIENT, [448, 40, 8], 520, 2056, (256, 256)),
    (FORWARD, [300, 0, 171], 391, 523, (128, 128)),             # no whole 16 bytes
    (ROW_GRADIENT, [30, 0, 17], 391, 523, (128, 128)),
    (ROW_GRADIENT, [300, 0, 171], 391, 524, (128, 128)),
    (WEIGHT_GRADIENT, [300, 0, 171], 391, 523, (128, 128)),
    (FOUR_BITS, [16, 0, 33, 1], 160, 640, (64, 128)),
    (FOUR_BITS, [130, 0, 257, 31], 288, 1152, (128, 128)),
    (FOUR_BITS, [4300, 4100], 1056, 640, (256, 256)),           # 2 steps and a half
    (FOUR_BITS, [4300, 4100], 1056, 1280, (256, 256)),          # 5
    (FOUR_BITS, [2600, 0, 5900], 1120, 2048, (256, 256)),       # 8
    (FOUR_BITS, [8400], 1056, 1152, (256, 256)),                # 4 and a half
    (FOUR_BITS, [8399], 1056, 128, (256, 256)),
]
