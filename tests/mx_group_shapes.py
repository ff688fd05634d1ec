"""Products grouped by rows that between them reach every tile shape of both activation kinds on 256 CUs: group sizes
with empty groups, a last tile of rows and of columns that is not full, and a K that ends inside a step."""

MANY = [12, 0, 37, 1, 70, 5, 33] * 10  # 70 groups
SOME = [0, 300, 12, 129, 60, 1, 91, 200] * 8

# (sizes of the groups, rows of W per group, K): activation kind, tile
GROUPED = [
    (([3, 0, 1, 30, 2, 0, 0, 5], 200, 96), "bf16", (32, 128)),
    (([60, 0, 33, 64, 1, 70, 9, 65], 6200, 1056), "bf16", (64, 128)),
    ((MANY[:56], 1400, 1056), "bf16", (32, 256)),
    ((MANY + [0, 641, 777], 1400, 1056), "bf16", (64, 256)),
    (([4000, 100, 0, 3991], 4600, 1056), "bf16", (128, 256)),
    (([3, 0, 1, 30, 2, 0, 0, 5], 200, 96), "mx", (64, 128)),
    (([150, 100, 0, 31, 257, 401, 0, 85], 2100, 1056), "mx", (128, 128)),
    ((SOME, 450, 1056), "mx", (128, 256)),
    (([4000, 100, 0, 3991], 4600, 1056), "mx", (256, 256)),
]
