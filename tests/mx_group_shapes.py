"""Products grouped by rows that between them reach every tile shape of both activation kinds on 256 CUs: group sizes
with empty groups, a last tile of rows and of columns that is not full, and a K that ends inside a step."""

# (sizes of the groups, rows of W per group, K): activation kind, tile
GROUPED = [
    (([3, 0, 1, 30, 2, 0, 0, 5], 200, 96), "bf16", (32, 128)),
    (([60, 0, 33, 64, 1, 70, 9, 65], 6200, 1056), "bf16", (64, 128)),
    (([14021, 0, 700, 1279], 202, 1056), "bf16", (128, 128)),
    (([1300, 100, 0, 391], 14600, 4128), "bf16", (128, 256)),
    (([4000, 100, 0, 3991], 14600, 1056), "bf16", (256, 256)),
    (([3, 0, 1, 30, 2, 0, 0, 5], 200, 96), "mx", (32, 128)),
    (([60, 0, 33, 64, 1, 70, 9, 65], 6200, 1056), "mx", (64, 128)),
    (([257, 100, 0, 391], 4600, 1056), "mx", (128, 128)),
    (([1000, 2000], 4000, 1056), "mx", (128, 256)),
    (([4000, 100, 0, 3991], 14600, 1056), "mx", (256, 256)),
]
