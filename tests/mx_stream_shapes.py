"""Products grouped by rows with MXFP4 activations that load W past the caches, between them in every tile shape that such a
product takes on 256 CUs: (sizes of the groups, rows of W per group, K), tile."""
STREAMED = [
    (([4000, 100, 0, 4000], 4608, 5600), (256, 256)),
    (([300, 0, 12, 129, 60, 1, 91, 200] * 8, 1152, 2080), (128, 256)),
    (([300, 0, 257, 20, 61, 1, 100, 161], 3136, 4128), (64, 128)),
    (([3, 0, 1, 30, 2, 0, 0, 5], 192, 96), (64, 128)),
]
