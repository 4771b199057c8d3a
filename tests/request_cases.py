"""Chunk calls whose sizes choose the kernel that a test is about: tests/test_request_plan_host.py
holds the choice to these lists, so that a change of the estimates fails there."""

# (dtype, rows of the sequences, their lengths, key heads, query heads per key head, D, window,
#  kernel, more than one split)
ODD = [
    ("f32", [2000], [2112], 1, 8, 64, 0, "tile", True),
    ("bf16", [2000], [2112], 1, 8, 64, 0, "tile", True),
    ("f16", [2000], [2112], 1, 8, 64, 0, "tile", True),
    ("f32", [4000], [4112], 1, 32, 64, 1500, "tile", False),
    ("bf16", [4000], [4112], 1, 32, 64, 1500, "tile", False),
    ("f16", [2000], [6000], 1, 16, 64, 900, "tile", False),
    ("bf16", [900], [3000], 1, 16, 128, 0, "tile", True),
    ("f32", [600], [3000], 1, 16, 80, 0, "tile", True),
    ("bf16", [600], [3000], 1, 16, 80, 0, "tile", True),
    ("f32", [500], [6000], 1, 16, 96, 0, "tile", True),
    ("f16", [500], [6000], 1, 16, 96, 0, "tile", True),
    ("bf16", [700], [3000], 1, 16, 256, 0, "tile", True),
    ("f16", [700], [3000], 1, 16, 200, 0, "tile", True),
    ("bf16", [700], [3000], 1, 16, 40, 0, "tile", True),
    ("f32", [1200], [3000], 1, 16, 32, 0, "tile", True),
    ("f16", [1200, 5], [3000, 2000], 2, 16, 32, 0, "tile", True),
    # the streaming kernel over more keys than it holds places of at once
    ("f32", [520], [2500], 8, 8, 256, 0, "stream", False),
    ("f32", [500, 3, 40], [2500, 2100, 2047], 8, 8, 200, 2000, "stream", False),
    # ... and over few
    ("bf16", [9], [130], 2, 1, 64, 0, "stream", False),
    ("f16", [40], [5000], 1, 4, 80, 0, "stream", True),
]

# (dtype, case of test_gpu_requests.test_chunk_attention): the tiled kernel in fp32, sequences
# with different numbers of rows among them
TILED = [
    ("f32", ([400, 1], [8100, 9000], 400, 32, 8, 96, 24, 0, "both")),
    ("f32", ([400, 113], [6100, 9000], 400, 32, 8, 96, 16, 0, "library")),
    ("f32", ([700, 0, 600], [2600, 7, 1900], 700, 32, 4, 64, 16, 0, "slots")),
]
# (dtype, n, query heads, key heads, D) of test_chunk_rows_that_do_not_exist
CUT = [("f32", 1000, 32, 8, 128)]
# (dtype, n, query heads, key heads, slots past 160) of the test of missing pages
MISSING = [("f32", 300, 32, 2, 992)]
# (dtype, case): the tiled kernel with few values per head, and with widths that fill its LDS rows
# by less than half
NARROW = [
    ("bf16", ([900], [2000], 900, 16, 1, 8, 16, 0, "library")),
    ("bf16", ([900], [2000], 900, 16, 1, 16, 8, 0, "slots")),
    ("f16", ([900], [2000], 900, 16, 1, 24, 16, 0, "both")),
    ("f32", ([2000], [2000], 2000, 16, 1, 16, 16, 0, "library")),
    ("bf16", ([900], [2000], 900, 16, 1, 136, 16, 0, "library")),
]
