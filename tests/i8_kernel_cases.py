"""Sizes that reach each kernel of the 8-bit products, for the tests that run
them and for the one that holds the sizes to the rules."""

# kernel, M, N: 16-byte aligned operands, then others
PRODUCTS = [
    ("stream 16x16", 16, 250), ("stream 16x16", 1, 4000), ("stream 16x32", 5, 8000), ("stream 32x32", 30, 8000),
    ("32x64", 40, 8000), ("64x64", 60, 16000), ("64x128", 500, 4000), ("128x128", 1000, 4000), ("128x256", 2000, 4000),
    ("ping-pong 256x256", 2050, 4100),
    # C narrower than the large tiles
    ("32x64", 3, 40000), ("64x128", 50, 40000), ("128x128", 40000, 100), ("128x256", 100, 70000),
]
PRODUCTS_UNALIGNED = [("unaligned stream 16x16", 40, 300), ("unaligned stream 32x32", 100, 1000), ("unaligned 32x32", 300, 1000),
                      ("unaligned 64x64", 1000, 1000), ("unaligned 128x128", 1500, 2100),
                      ("unaligned 128x256", 2000, 4000)]

_GRADIENTS = [("stream 32x32", 100, 200), ("stream 32x64", 500, 600), ("64x64", 1000, 1000), ("64x128", 1000, 2000),
              ("128x128, deep", 2000, 2000)]


def gradients(wide, split_a, aligned):
    """wide: fp32 C; split_a: of fp16 or fp32 A."""
    if split_a:
        more = [("64x128", 2304, 1950), ("128x256", 2600, 1950)] if aligned else [("64x128, two a CU", 2304, 1950)]
    elif not aligned:
        more = [("128x128", 2304, 1950)]
    elif wide:
        more = [("128x128", 2304, 1950), ("256x128", 2600, 1950)]
    else:
        more = [("128x128", 2304, 1950), ("256x256", 3300, 3100), ("64x64", 40000, 40), ("128x128", 100, 50000)]
    return _GRADIENTS + more


# aligned, M, N, K; rows and columns at the end that a call of their own computes
EDGES = [(True, 2049, 4100, 2048, 1, 4), (True, 2053, 4096, 2048, 5, 0), (True, 2048, 4112, 2047, 0, 16),
         (False, 2050, 4100, 1501, 2, 4), (False, 2048, 4100, 1501, 0, 4), (True, 2060, 4110, 1041, 0, 0)]
