"""Sizes that take each form of the weight streams (csrc/skinny.h): items of 64 rows and of several times 64,
beside those whose k's the waves split, over experts of every number of columns. Which form a case takes is
checked against the launch rule itself on the host (test_stream_forms.py); test_streams_gpu.py runs them."""

# pairs of the first experts: one pass of 4, 8, 16, 32 and 64 columns, and several passes; the others have one
POPULAR = (3, 7, 13, 29, 50, 70, 130)

# 4-bit product: E, N, block_m, K by group, and the form (split, tiles)
PRODUCT = [
    (130, 200, 64, {32: 256, 64: 256, 128: 256}, (0, 1)),
    (130, 200, 200, {32: 672, 64: 704, 128: 640}, (0, 1)),      # blocks of several passes; rows of 6 loads
    (130, 200, 64, {32: 2304, 64: 2304, 128: 2304}, (0, 1)),    # x in several stages at every width
    (260, 200, 64, {32: 768, 64: 768, 128: 768}, (0, 2)),
    (260, 199, 200, {32: 1536, 64: 1536, 128: 1536}, (0, 2)),   # one stage up to 8 columns, several beyond
    (520, 200, 64, {32: 384, 64: 384, 128: 384}, (0, 4)),
    (520, 201, 64, {32: 736, 64: 704, 128: 768}, (0, 4)),
    (9, 200, 200, {32: 736, 64: 704, 128: 768}, (1, 1)),        # split, passes of 8
]

# layer: dtype, group, E, hidden, inter, and the forms of gate/up and down
LAYER = [
    ("bf16", 0, 130, 256, 128, (0, 1), (0, 1)), ("f32", 0, 130, 260, 132, (0, 1), (0, 1)),
    ("bf16", 0, 130, 1152, 520, (0, 1), (0, 1)), ("f32", 0, 130, 1152, 260, (0, 1), (0, 1)),
    ("bf16", 0, 270, 264, 120, (0, 2), (0, 4)), ("bf16", 0, 530, 136, 96, (0, 4), (0, 4)),
    ("bf16", 0, 530, 256, 72, (0, 2), (0, 4)), ("f32", 0, 530, 132, 68, (0, 2), (0, 4)),
    ("bf16", 32, 130, 256, 160, (0, 1), (0, 1)), ("bf16", 64, 130, 704, 192, (0, 1), (0, 2)),
    ("bf16", 128, 130, 768, 640, (0, 4), (0, 2)), ("bf16", 128, 130, 2304, 128, (0, 1), (0, 4)),
    ("bf16", 32, 130, 1152, 544, (0, 2), (0, 4)), ("bf16", 64, 130, 1152, 1088, (0, 2), (0, 2)),
    ("bf16", 32, 530, 256, 96, (0, 4), (0, 4)), ("bf16", 64, 530, 256, 128, (0, 4), (0, 4)),
    ("bf16", 128, 530, 256, 128, (0, 4), (0, 4)), ("f32", 32, 130, 288, 160, (0, 1), (0, 1)),
    ("f32", 64, 530, 256, 128, (0, 4), (0, 4)), ("f32", 128, 130, 1152, 640, (0, 2), (0, 4)),
]

# layer, fewer pairs than experts (96 of 130): dtype, group, hidden, inter, forms
BY_PAIR = [
    ("bf16", 0, 1024, 512, (0, 1), (0, 1)), ("bf16", 32, 1024, 512, (0, 2), (0, 2)),
    ("bf16", 64, 1024, 512, (0, 2), (0, 2)), ("bf16", 128, 1024, 768, (0, 2), (0, 2)),
    ("f32", 0, 512, 260, (0, 1), (0, 1)), ("f32", 64, 512, 256, (0, 1), (0, 1)),
]


def product_pairs(E):
    """Experts of the pairs of a product case, in an order that mixes them."""
    one = [e for e in range(len(POPULAR), E)]
    return one + [e for j in range(max(POPULAR)) for e, n in enumerate(POPULAR) if j < n]
