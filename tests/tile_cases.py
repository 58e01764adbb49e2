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
