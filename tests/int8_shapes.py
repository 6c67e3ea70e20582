"""Shapes of int8 products and the kernel that each is there for, with rows that start at lines of memory (128
bytes) or anywhere: what the choice of kernels makes of them is checked on the CPU, their results on the GPU."""

LINE, ANY = 128, 16

# M, N, K, where rows start: tiles of 256 x 256 in one to three rounds of 256 workgroups, all of them cut off at
# the last rows and columns, with columns that are a multiple of four and not; and in front of smaller tiles
WIDE = [
    (1154, 10784, 1922, LINE, "256x256"),
    (5458, 5708, 937, LINE, "256x256"),
    (3925, 11844, 523, LINE, "256x256"),
    (4062, 7760, 1180, ANY, "256x256"),
    (7196, 6364, 808, ANY, "256x256"),
    (3731, 8290, 2192, LINE, "256x256"),
    (7865, 6129, 1795, LINE, "256x256"),
    (2988, 6440, 777, LINE, "256x256 128x128"),
    (5270, 3564, 791, ANY, "256x256 128x128"),
]
TILES = [
    (132, 11469, 552, LINE, "128x128"), (11796, 135, 535, ANY, "128x128"),
    (11445, 267, 508, LINE, "128x192"), (269, 10922, 594, ANY, "128x192"),
    (263, 11197, 623, LINE, "192x128"), (273, 11154, 563, ANY, "192x128"),
    (11090, 543, 508, LINE, "192x192"), (790, 7248, 539, ANY, "192x192"),
    (831, 6925, 500, LINE, "128x256"), (8107, 1018, 720, ANY, "128x256"),
    (7161, 793, 511, LINE, "256x128"), (13000, 630, 720, ANY, "256x128"),
    (9040, 73, 500, LINE, "64x128"), (68, 9333, 580, ANY, "64x128"),
    (200, 333, 1248, LINE, "64x64"), (153, 205, 700, ANY, "64x64"),
    (8863, 2094, 1451, ANY, "128x192 cut"), (9954, 1841, 1821, ANY, "192x192 cut"),
    (9, 700, 700, ANY, "few"), (27, 333, 1000, LINE, "few"),
]


def pitch(K, start):
    return -(-K // start) * start
