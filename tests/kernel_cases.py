"""Sizes for single kernels of the training and 8-bit calls, each with the choice
(tests/kernel_rules.py) that it is there for.  Segment lengths and expected lengths
(T k / E, which the rules see) are independent of each other."""
from tests.kernel_rules import WG_LONG, WG_SHORT, WG_SPLIT
from tests.segments import spec

# lengths around the 64-row stages of the weight gradients: none, part of a stage,
# one, two, an odd number of them, many
MIXED = [0, 7, 64, 65, 128, 129, 200, 1, 0, 255, 192, 33]


def _mixed(n):
    return [MIXED[(5 * e + e // 12) % 12] for e in range(n)]


# name: (counts, d, f, spec arguments, what the plan says: fields of Train and Backward)
TRAINING = {
    # rows of 4 KB: the input gradient starts at other K stages and wraps around, over
    # both of its products
    "rotated_64": ([5, 130, 1, 0, 257, 0], 264, 2048, {}, dict(input=1, mode=WG_SHORT)),
    "rotated_128": ([(150 + 7 * e) // (1 + e % 3) for e in range(33)], 40, 2048, dict(T=424, k=32), dict(input=2, mode=WG_SHORT)),
    "rotated_192": ([60 + 2 * e * (e % 4) for e in range(70)], 40, 2048, dict(T=960, k=32), dict(input=3, mode=WG_SHORT)),
    "rotated_split": ([700, 901], 40, 2048, dict(T=2014, k=1, E=4), dict(input=1, mode=WG_SPLIT)),
    "rotated_long": ([0, 555, 1001], 40, 2048, dict(T=1104, k=2, E=4), dict(input=1, mode=WG_LONG)),
    "rotated_8k": ([5, 70, 0, 300], 72, 4096, {}, dict(input=1)),
    # units of several row blocks that share their columns, the last unit shorter
    "units_of_2": (_mixed(70), 1080, 288, dict(T=255, k=32), dict(mode=WG_SHORT, div=2, input=3)),
    "units_of_2_narrow": (_mixed(140), 1200, 72, dict(T=500, k=32, E=512), dict(mode=WG_SHORT, div=2)),
    "units_of_3": (_mixed(130), 1800, 72, dict(T=500, k=32, E=512), dict(mode=WG_SHORT, div=3)),
    "units_of_4": (_mixed(171), 1944, 40, dict(T=500, k=32, E=1024), dict(mode=WG_SHORT, div=4)),
    # every height of the input gradient beside long and split weight gradients
    "long_64": ([1000], 264, 824, dict(T=1028, k=1, E=2), dict(input=1, mode=WG_LONG)),
    "long_128": ([518, 0, 300, 517, 1, 64, 63, 65, 500], 440, 56, dict(T=518, k=9), dict(input=2, mode=WG_LONG)),
    "split_128": ([1000, 0, 2500, 17, 640, 64, 1], 48, 48, dict(T=4744, k=4, E=8), dict(input=2, mode=WG_SPLIT)),
    "split_192": ([2000 - 150 * e for e in range(13)], 56, 48, dict(T=2790, k=13), dict(input=3, mode=WG_SPLIT)),
    "split_256": ([1214 - 38 * e for e in range(32)] + [0], 48, 80, dict(T=1252, k=32), dict(input=4, mode=WG_SPLIT)),
}

# name: (counts, d, f, spec arguments, fields of the gated product's plan, of the down projection's)
QUANTIZED = {
    # one launch: segments of up to 128 rows in blocks of 32
    "blocks": ([0, 128, 33], 1048, 976, dict(T=128, k=2, E=24), dict(stream=1, tiles=0, wide=0, low=0, blocks=4),
               dict(stream=1, tiles=0, wide=0, low=0, blocks=4)),
    "blocks_four": ([128, 1, 70, 32], 976, 976, dict(T=128, k=2, E=32), dict(stream=1, tiles=0, wide=0, low=0, blocks=4),
                    dict(stream=1, tiles=0, wide=0, low=0, blocks=4)),
    "blocks_wide": ([(29 * e) % 122 if e % 3 else 0 for e in range(16)], 976, 616, dict(T=121, k=8, E=512),
                    dict(stream=1, tiles=0, wide=1, low=0, blocks=4), dict(stream=1, tiles=0, wide=1, low=0, blocks=4)),
    # two launches: segments of up to 32 rows stream, longer ones take tiles
    "split": ([0, 5, 33, 130, 1, 257], 4096, 512, dict(T=257, k=2, E=48), dict(stream=1, tiles=1, wide=0), dict(stream=0)),
    "split_down": ([20, 300, 33], 24, 4600, dict(T=542, k=1, E=24), dict(stream=0), dict(stream=1, tiles=1, wide=0)),
    "split_both": ([32, 257, 0, 7, 33, 1, 64, 200], 4192, 40, dict(T=300, k=4, E=64), dict(stream=1, tiles=1, wide=0),
                   dict(stream=1, tiles=1, wide=1)),
    "split_wide": ([(37 * e) % 41 if e % 9 else (43 * e) % 300 for e in range(100)], 400, 184, dict(T=1500, k=3, E=800),
                   dict(stream=1, tiles=1, wide=1), dict(stream=1, tiles=1, wide=1)),
    # batches of up to 16 tokens
    "low": ([4, 0, 16, 1], 976, 976, dict(T=16, k=4), dict(stream=1, wide=0, low=1), dict(stream=1, wide=0, low=1)),
    "low_wide": ([e % 4 for e in range(64)], 328, 112, dict(T=6, k=32, E=64), dict(stream=1, wide=1, low=1),
                 dict(stream=1, wide=1, low=1)),
}

# gemm_quantized: (rows, columns, K), plan
PRODUCTS = {
    "low": ((16, 24, 8208), dict(stream=1, wide=0, low=1)),
    "low_wide": ((3, 16520, 400), dict(stream=1, wide=1, low=1)),
    "blocks": ((250, 24, 8208), dict(stream=1, wide=0, low=0, blocks=8)),
    "blocks_wide": ((70, 16520, 400), dict(stream=1, wide=1, low=0, blocks=3)),
    "tiles_64": ((300, 520, 400), dict(stream=0, height=1)),
    "tiles_128": ((2049, 2104, 80), dict(stream=0, height=2)),
    "tiles_192": ((1995, 4320, 208), dict(stream=0, height=3)),
    "tiles_256": ((4096, 4096, 208), dict(stream=0, height=4)),
}


def problem(case, dtype="bf16"):
    counts, d, f, kw = case[:4]
    assert all(0 <= c <= kw.get("T", c) for c in counts)
    return spec(counts, d, f, dtype, **kw)
