"""Sizes (rows, in, out) of 4-bit products that together reach every kernel
instance and path that the dispatch picks at real sizes."""

FORMS = [
    # up to 16 rows: 32 weight rows of a block, with remainders along rows, inputs and outputs
    (1, 4096, 4100), (8, 4192, 4096), (13, 4128, 4113),
    # and 16 of them
    (2, 4096, 4088), (16, 2880, 5121),
    # 17 to 128 rows: a CTA along K, two, three and four; rings that wrap; outputs that are no
    # multiple of 8; inputs that leave 32, 64 and 96 of a block; one tile of tokens and two
    (40, 1056, 9801), (128, 2144, 5000), (40, 1440, 6600), (30, 2144, 6001), (17, 4064, 4097), (20, 8192, 130), (70, 1056, 201),
    (24, 96, 77), (33, 224, 1001), (128, 2880, 1033),
    # above: both of the dense products' kernels
    (129, 288, 1001), (300, 512, 2048), (257, 2880, 1033),
]
