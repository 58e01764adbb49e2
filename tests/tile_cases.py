"""Sizes at which the planner takes its larger tiles, each with the tile it is to take (256 compute units): run on the GPU by
test_gpu_tiles.py, and held to the planner on the host by test_planned_tiles.py, so that none of them can fall back to
smaller tiles unseen."""

# Grouped weight gradients.  name: (tokens of each expert, N, K, tile rows, whether a workspace lets experts be split)
WGRAD = {
    "whole": ([600, 1, 0, 300, 450], 2048, 1408, 256, False),
    "split": ([9000, 500, 0, 3], 2048, 1408, 256, True),
    "even": ([300] * 16, 1024, 768, 256, False),
    "middle": ([3000, 2000, 0, 1], 512, 768, 128, False),
}


def padded(counts):
    T, E = sum(counts), len(counts)
    return (T + 127 * min(E, T)) // 128 * 128


# Grouped fprop and dgrad.  name: (tokens of each expert, N, K, tile rows of fprop, of dgrad).  The experts' last tiles hold 1,
# 128, 129 and 255 rows, or experts have as many in all; some have none.
ROWS = {
    "middle": ([700, 1, 0, 255, 513, 384, 640], 2048, 1408, 128, 128),
    "tall": ([513, 385, 0, 255, 384] * 7, 1024, 512, 256, 128),
    "tall_dgrad": ([513, 385, 0, 255, 384] * 7, 512, 1024, 128, 256),
    "tall_odd_width": ([700] * 12 + [1, 0, 129, 255], 1408, 512, 256, 128),
    "wide": ([1500, 0, 257, 129, 1280, 256], 2816, 512, 256, 64),
}

# Grouped MXFP4 products, widths that end inside a tile.  name: (tokens of each expert, N, K, tile rows)
MX_GROUPED = {
    "middle": ([700, 1, 0, 255, 513, 384, 640], 1992, 1440, 128),
    "middle_odd": ([513, 385, 0, 255, 384] * 7, 493, 1056, 128),
    "tall": ([1500, 0, 257, 129, 1280, 256], 2760, 512, 256),
    "tall_odd": ([1500, 0, 257, 129, 1280, 256], 2797, 544, 256),
}

# MXFP4 products whose contraction is split over workgroups.  (M, N, K, tile rows, parts)
MX_SPLIT = [(64, 2048, 11264, 64, 8), (77, 130, 8224, 64, 7), (200, 72, 16416, 64, 8), (300, 1001, 11296, 64, 5),
            (512, 512, 16384, 64, 6), (900, 1001, 11296, 128, 4), (1100, 1100, 16416, 128, 4), (2429, 1032, 24608, 256, 4)]
