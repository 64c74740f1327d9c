"""Sizes of the tests of E4M3 rows: rows, outputs, columns.  Between them they reach every kernel that makes such rows or sums for
them, split and unsplit, with weights read once or again and outputs that end inside a block of 128."""

E4M3_ROWS = [
    (1, 16, 128), (7, 144, 272), (3, 4112, 400), (32, 4112, 400), (5, 1040, 4112), (33, 16, 16), (12, 1024, 4096), (64, 128, 256), (48, 1408, 1040), (100, 272, 400),
    (257, 400, 1040), (300, 1040, 528), (16, 1408, 4096), (64, 1408, 4096), (200, 1408, 4096), (150, 1040, 4112), (700, 4000, 400),
    (600, 8208, 144), (72, 10464, 1088), (261, 896, 80), (500, 4112, 1040), (1000, 1424, 4096), (1100, 1424, 2064), (40, 8208, 4096), (2, 11008, 4096), (1, 13824, 5120), (48, 13824, 5120),
]
