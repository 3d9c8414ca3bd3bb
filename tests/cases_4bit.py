"""Sizes of 4-bit products, named by the kernels they are there for: (sizes, what the
library's rules say of them).  tests/test_4bit_choice.py holds the two together."""

# M, K, N, group; what tests/rules_4bit.py's plan has
PRODUCTS = {
    "narrow, 16 rows": ((5, 136, 24, 32), dict(tiles=False, wide=False, low=True, waves=8)),
    "narrow, long": ((9, 4104, 72, 64), dict(tiles=False, wide=False, low=True, waves=16)),
    "narrow, 32 rows": ((24, 520, 40, 128), dict(tiles=False, wide=False, low=False, blocks=1)),
    "narrow, blocks of rows": ((50, 2056, 136, 64), dict(tiles=False, wide=False, low=False, blocks=2)),
    "wide, 16 rows": ((7, 264, 8200, 128), dict(tiles=False, wide=True, low=True, ahead=False, waves=8)),
    "wide, 32 rows": ((30, 392, 8200, 32), dict(tiles=False, wide=True, low=False, ahead=False, waves=4)),
    "wide, 16 rows, a block ahead": ((6, 1032, 8200, 64), dict(tiles=False, wide=True, low=True, ahead=True, waves=4)),
    "wide, 32 rows, a block ahead": ((20, 1160, 8200, 32), dict(tiles=False, wide=True, low=False, ahead=True, waves=4)),
    "wide, blocks of rows": ((100, 264, 1032, 64), dict(tiles=False, wide=True, low=False, blocks=4)),
    "tiles of 64, one block": ((1092, 8, 2056, 32), dict(tiles=True, bm=64, parts=1)),
    "tiles of 64": ((286, 520, 8200, 128), dict(tiles=True, bm=64, parts=1)),
    "tiles of 128 and 64": ((1030, 136, 4104, 64), dict(tiles=True, bm=128, parts=1)),
    "tiles of 128 and 96": ((472, 520, 8200, 32), dict(tiles=True, bm=128, parts=1)),
    "tiles of 192 and 160": ((906, 264, 8200, 64), dict(tiles=True, bm=192, parts=1)),
    "tiles of 192 and 64": ((968, 136, 8200, 128), dict(tiles=True, bm=192, parts=1)),
    "tiles of 192 and 96": ((1030, 264, 8200, 32), dict(tiles=True, bm=192, parts=1)),
    "tiles of 192 and 128": ((1061, 136, 8200, 64), dict(tiles=True, bm=192, parts=1)),
    "K in parts, 64 rows": ((130, 14344, 136, 64), dict(tiles=True, bm=64, parts=15, per=8)),
    "K in parts, 128 rows": ((355, 14344, 520, 128), dict(tiles=True, bm=128, parts=15, per=8)),
    "K in parts, 96 rows": ((330, 14344, 520, 32), dict(tiles=True, bm=128, parts=15, per=8)),
}

# rows of the experts, d, f, group; plans of the gated product and of the other
EXPERTS = {
    "streams": (([40, 30, 50, 64, 7, 30, 0, 60], 136, 264, 64), dict(tiles=False), dict(tiles=False)),
    "tiles of every height": (([60, 90, 120, 150, 190, 250, 0, 33], 392, 2056, 128), dict(tiles=True, bm=192), dict(tiles=False)),
    "groups of 32": (([60, 90, 120, 150, 190, 250, 0, 33], 136, 2056, 32), dict(tiles=True, bm=192), dict(tiles=False)),
    "both tiles": (([150, 20, 155, 0, 130, 260, 96, 200], 2056, 2056, 64), dict(tiles=True, bm=192), dict(tiles=True, bm=64)),
    "tiles of 128": (([190, 120, 300, 140, 130, 170, 100, 160], 136, 1032, 64), dict(tiles=True, bm=128), dict(tiles=False)),
    "tiles of 64": (([150, 20, 155, 0, 130, 260, 96, 200], 136, 1032, 128), dict(tiles=True, bm=64), dict(tiles=False)),
    "down alone": (([190, 120, 300, 140, 130, 170, 100, 160], 2056, 136, 32), dict(tiles=False), dict(tiles=True, bm=128)),
}
