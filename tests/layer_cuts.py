"""Products that reach every cut of the matrix products: sizes that end
inside a tile on every side, with the cut and the splits of the depth that the
library takes for them. The CPU tests pin the cuts, the GPU tests run them."""

# names in the order of arx_shapes.h's enum
NAMES = ("rows16", "rows32", "64x64", "64x128", "128x128", "256x256")

# (rows, columns, depth): cut, splits; the same in the three layouts and with
# sizes rounded up to multiples of eight, which the tiles load as they lie.
# Depths of one step, of a few, and of more than a tile's buffers hold.
TILES = {
    (33, 42, 61): ("64x64", 1), (70, 77, 143): ("64x64", 1), (130, 333, 491): ("64x64", 1),
    (333, 777, 1001): ("64x64", 1), (70, 130, 3663): ("64x64", 8), (200, 260, 8203): ("64x64", 8),
    (67, 8551, 61): ("64x128", 1), (8514, 67, 142): ("64x128", 1), (66, 8291, 461): ("64x128", 1),
    (143, 5651, 2435): ("64x128", 3),
    (259, 6609, 61): ("128x128", 1), (193, 8302, 131): ("128x128", 1), (7195, 387, 458): ("128x128", 1),
    (1021, 1030, 4101): ("128x128", 3),
    (1314, 8834, 61): ("256x256", 1), (7500, 1025, 129): ("256x256", 1), (2049, 4100, 1203): ("256x256", 1),
    (5562, 157, 5598): ("256x256", 8),
}

# (m, n, k) of few rows: the cut and splits on 16-byte boundaries, and off them
ROWS = {
    (1, 4096, 2048): (("rows16", 1), ("rows16", 1)), (3, 41, 70): (("rows16", 1), ("rows16", 1)),
    (16, 1025, 4100): (("rows16", 3), ("rows16", 3)), (5, 300, 16387): (("rows16", 8), ("rows16", 8)),
    (15, 2055, 8190): (("64x64", 6), ("rows16", 1)),
    (17, 1024, 1024): (("rows32", 1), ("64x64", 4)), (32, 40, 72): (("rows32", 1), ("64x64", 1)),
    (32, 700, 4096): (("rows32", 4), ("64x64", 8)), (20, 513, 16384): (("rows32", 6), ("64x64", 8)),
}

# (m, n, k) of a backward pass whose two products take one launch: whether the
# weight's tiles come first
PAIRS = {(351, 332, 5674): True, (1030, 1025, 2000): True, (600, 520, 5000): True,
         (330, 408, 5455): False, (2050, 2056, 1000): False, (336, 408, 5456): False}


def up8(n):
    return (n + 7) // 8 * 8


def in_layout(size, layout, as_is):
    """size with what has to be a multiple of eight rounded up where the tiles
    load the operands as they lie. fwd: both depth-contiguous; dx: the right
    operand's rows contiguous; dw: both."""
    m, n, k = size
    if not as_is:
        return size
    return {"fwd": (m, n, up8(k)), "dx": (m, up8(n), up8(k)), "dw": (up8(m), up8(n), k)}[layout]
