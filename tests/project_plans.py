"""Sizes of 4-bit products, rows x columns of depth, that between them take every way through the kernels, and the way of each: the
width of its tiles (or of the MMAs of few rows), the parts of its depth, the most tiles that a pair of SMs takes one after another."""

FEW = {
    (3, 200, 2048): (16, 1, 1), (3, 10000, 3200): (16, 2, 1), (3, 300, 3200): (16, 4, 1), (16, 257, 9000): (16, 8, 1),
    (17, 1000, 1100): (32, 1, 1), (17, 10000, 3200): (32, 2, 1), (31, 1030, 3330): (32, 4, 1), (32, 513, 4096): (32, 8, 1),
    (40, 130, 2048): (64, 1, 1), (64, 10000, 3200): (64, 2, 1), (40, 300, 3200): (64, 4, 1), (64, 300, 7001): (64, 8, 1),
}
TILES = {
    (70, 300, 2048): (128, 1, 1), (4100, 1600, 300): (128, 1, 3), (700, 650, 8300): (128, 2, 1), (77, 4100, 8200): (128, 2, 1),
    (90, 260, 9000): (128, 4, 1), (1560, 1530, 700): (192, 1, 1), (4500, 1530, 1300): (192, 1, 2), (2040, 2050, 300): (256, 1, 1),
    # pairs' later tiles of 256: whole rows and rows that TMA cannot write, tiles of a or of b varying fastest, the last round not full
    (5400, 2500, 300): (256, 1, 3), (5400, 2501, 300): (256, 1, 3), (1500, 8000, 1300): (256, 1, 3), (4680, 6144, 1536): (256, 1, 6),
}
PLANS = {**FEW, **TILES}
