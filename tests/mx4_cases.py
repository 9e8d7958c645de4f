"""Sizes that take each form of the product over microscaled 4-bit weights (csrc/moe_mx4.h). Which form a case takes is
checked against the launch rule itself on the host (test_mx4_forms.py); test_moe_mx4_gpu.py runs them."""

SPLIT, NARROW, WIDE, SPREAD = 0, 1, 2, 3

# rows of x, M, E, topk, K, N, block_m, form
FORMS = [
    # narrow and spread: passes of 16, 32 and 64 columns and several of them, one stage of x and several, more k's than the scales of
    # x that are staged at a time
    ("codes", 40, 40, 1, 96, 130, 64, NARROW), ("codes", 100, 5, 1, 1056, 65, 64, NARROW),
    ("codes", 150, 3, 1, 2592, 67, 64, NARROW), ("codes", 130, 2, 1, 4160, 64, 200, SPREAD),
    ("codes", 700, 3, 1, 4128, 100, 1024, SPREAD),
    ("bf16", 40, 40, 1, 96, 130, 64, NARROW), ("bf16", 100, 5, 1, 1056, 65, 64, SPREAD),
    ("bf16", 150, 3, 1, 2592, 67, 64, SPREAD), ("bf16", 700, 3, 1, 1056, 100, 1024, SPREAD),
    ("codes", 130, 2, 1, 2592, 12301, 200, SPREAD), ("bf16", 130, 2, 1, 1056, 12301, 200, SPREAD),
    ("bf16", 300, 290, 1, 96, 290, 64, NARROW), ("codes", 90, 2, 1, 288, 700, 96, SPREAD), ("bf16", 90, 2, 1, 288, 700, 48, SPREAD),
    ("f32", 600, 300, 1, 96, 130, 64, NARROW), ("f32", 900, 100, 1, 1056, 190, 64, NARROW),
    # fp32 rows, split k's: one pass of 16 columns and several, fewer units than waves, and more stages than one
    ("f32", 5, 2, 1, 32, 17, 16, SPLIT), ("f32", 30, 3, 2, 416, 100, 64, SPLIT), ("f32", 60, 2, 1, 2144, 40, 64, SPLIT),
    # wide: K of one unit, of a part of one, of more than the staged scales; odd numbers of rows; spans of a block
    ("codes", 1000, 2, 1, 32, 6401, 128, WIDE), ("codes", 1000, 2, 1, 256, 6400, 128, WIDE),
    ("codes", 1000, 2, 1, 288, 6461, 48, WIDE), ("codes", 900, 3, 1, 768, 6420, 200, WIDE),
    ("codes", 700, 2, 1, 2080, 7401, 128, WIDE), ("codes", 700, 2, 1, 4672, 6430, 1024, WIDE),
    ("codes", 3000, 60, 2, 352, 300, 128, WIDE),
    # wide over small blocks, two, four and eight of one expert together, the last of them partly filled; chains of
    # them past a wave's lanes; not over the smallest, nor for fp32 rows
    ("codes", 1000, 2, 1, 160, 6401, 64, WIDE), ("codes", 1500, 3, 1, 288, 4400, 32, WIDE),
    ("codes", 1000, 3, 1, 64, 5500, 16, WIDE), ("codes", 500, 2, 1, 64, 9000, 1, NARROW),
    ("codes", 1000, 3, 1, 96, 2500, 16, WIDE), ("codes", 500, 60, 4, 64, 1000, 16, WIDE),
    ("bf16", 1500, 3, 1, 160, 4400, 64, WIDE), ("bf16", 9000, 1, 1, 96, 700, 16, WIDE),
    ("f32", 700, 2, 1, 96, 130, 16, SPLIT),
    ("bf16", 1000, 2, 1, 32, 6401, 128, WIDE), ("bf16", 1000, 2, 1, 256, 6400, 128, WIDE),
    ("bf16", 1000, 2, 1, 288, 6461, 48, WIDE), ("bf16", 700, 2, 1, 2208, 6430, 1024, WIDE),
    ("bf16", 3000, 60, 2, 352, 300, 128, WIDE),
    ("f32", 300, 2, 1, 288, 130, 128, WIDE), ("f32", 200, 2, 1, 2208, 65, 1024, WIDE),
]
# narrow, and run with some popular experts, whose blocks take several passes
POPULAR = [(x, 600, 100, 4, K, 1300, 128, NARROW) for x in ("codes", "bf16") for K in (160, 2336)]
