"""Shapes of fp4_matmul and fp4_matmul_grad that reach every kernel there is (test_fp4_matmul_plan.py asks the library's plan
whether they still do)."""

# (format, x, gradient, batch, m, n, k): tiles of 16, 32, 64, 128 and 256 rows, each with and without its steps shared, as far
# as the plan shares them; rows, outputs and sums that end inside a tile, widths that end inside a thread's codes
TILES = [
    ("nvfp4", "bf16", False, 1, 1, 3311, 10160), ("mxfp4", "bf16", False, 1, 1, 4571, 7552), ("nvfp4", "f32", False, 1, 1, 3085, 6960), ("nvfp4", "bf16", False, 1, 1, 3311, 10176),
    ("mxfp4", "f32", False, 1, 1, 5593, 4064), ("nvfp4", "bf16", True, 1, 1, 1512, 4160), ("nvfp4", "bf16", True, 1, 1, 4099, 5136),
    ("mxfp4", "bf16", True, 1, 1, 1337, 8384), ("nvfp4", "f32", True, 1, 1, 977, 7248), ("mxfp4", "f32", True, 1, 1, 972, 6496),
    ("mxfp4", "bf16", False, 1, 17, 6517, 11264), ("nvfp4", "f32", False, 1, 27, 4623, 11952), ("mxfp4", "f32", False, 1, 19, 5205, 9792),
    ("nvfp4", "f32", True, 1, 18, 10960, 8816), ("mxfp4", "f32", True, 1, 17, 9270, 9984),
    ("nvfp4", "bf16", False, 1, 913, 3458, 288), ("nvfp4", "bf16", False, 1, 1500, 5003, 1040), ("nvfp4", "bf16", False, 1, 73, 5253, 8208),
    ("mxfp4", "bf16", False, 1, 2527, 1293, 288), ("mxfp4", "bf16", False, 1, 65, 8267, 4288), ("nvfp4", "f32", False, 1, 3408, 1008, 272),
    ("nvfp4", "f32", False, 1, 3300, 65, 6784), ("mxfp4", "f32", False, 1, 2161, 1685, 288), ("mxfp4", "f32", False, 1, 2173, 230, 4512),
    ("nvfp4", "bf16", True, 1, 423, 312, 7680), ("nvfp4", "bf16", True, 1, 75, 6546, 7984), ("mxfp4", "bf16", True, 1, 662, 269, 4800),
    ("mxfp4", "bf16", True, 1, 67, 10870, 4512), ("nvfp4", "f32", True, 1, 1177, 281, 2816), ("nvfp4", "f32", True, 1, 66, 6946, 3808),
    ("mxfp4", "f32", True, 1, 544, 261, 7072), ("mxfp4", "f32", True, 1, 82, 1434, 8576),
    ("nvfp4", "bf16", False, 1, 2628, 4178, 272), ("nvfp4", "bf16", False, 1, 2048, 4099, 656), ("nvfp4", "bf16", False, 1, 207, 9840, 7088),
    ("mxfp4", "bf16", False, 1, 1681, 5060, 288), ("mxfp4", "bf16", False, 1, 2719, 656, 7936), ("nvfp4", "f32", False, 1, 1176, 7888, 304),
    ("nvfp4", "f32", False, 1, 129, 4962, 7520), ("mxfp4", "f32", False, 1, 1849, 4542, 320), ("mxfp4", "f32", False, 1, 140, 4828, 6848),
    ("nvfp4", "bf16", True, 1, 1559, 330, 5584), ("nvfp4", "bf16", True, 1, 2100, 1001, 4112), ("nvfp4", "bf16", True, 1, 220, 10805, 6080),
    ("mxfp4", "bf16", True, 1, 3412, 259, 2560), ("mxfp4", "bf16", True, 1, 154, 6660, 9088), ("nvfp4", "f32", True, 1, 1787, 284, 5056),
    ("nvfp4", "f32", True, 1, 140, 3377, 9040), ("mxfp4", "f32", True, 1, 3497, 297, 2336), ("mxfp4", "f32", True, 1, 144, 3380, 9504),
    ("nvfp4", "bf16", False, 3, 1000, 1300, 1040), ("mxfp4", "f32", True, 2, 1100, 450, 2336), ("nvfp4", "bf16", True, 3, 70, 2001, 3600),
    ("nvfp4", "bf16", False, 1, 101, 35, 368), ("mxfp4", "f32", False, 1, 204, 61, 384), ("nvfp4", "f32", True, 1, 9, 331, 80),
    ("mxfp4", "bf16", True, 1, 30, 996, 96),
    ("nvfp4", "bf16", False, 1, 100, 70, 2064), ("mxfp4", "bf16", False, 1, 100, 70, 2080), ("mxfp4", "f32", False, 1, 150, 70, 2080),
    ("nvfp4", "f32", False, 1, 150, 70, 272), ("nvfp4", "bf16", True, 1, 9, 200, 80), ("mxfp4", "f32", True, 1, 9, 258, 32),
    ("mxfp4", "f32", True, 1, 100, 459, 96),
]

# (format, x, m, n, k) of the few-rows kernel: K of one, two and four steps a wave, in whole pieces of DMA and not
FEW = [(fmt, x, m, n, k)
       for fmt, ks in (("nvfp4", (1488, 1536, 2416, 2432, 3568, 3584, 5008, 5056, 7152, 7168)), ("mxfp4", (1504, 1536, 2400, 2432, 3552, 3584, 5024, 4992, 7136, 7168)))
       for k in ks for x, m, n in (("bf16", 3, 261), ("bf16", 20, 190), ("bf16", 50, 77), ("bf16", 64, 333), ("f32", 13, 100), ("f32", 128, 75))
       if x == "bf16" or k <= 3584]
