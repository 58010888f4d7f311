"""Sizes that reach each kernel of the grouped and adapter products, for the
tests that run them and for the one that holds the sizes to the rules.

Widths are multiples of 8 (16-byte rows of 16-bit elements) but of no tile;
`pad` 1 makes operands that are not 16-byte aligned.
"""

# kernel, by type, padding: groups' rows, N
ROWS_16 = [
    ("rows 32x64", [5, 0, 17, 3], 136, "kn"),
    ("rows 32x64", [16, 9, 0, 31] * 20, 504, "k"),
    ("rows 64x128", [16, 9, 0, 31] * 20, 504, "n"),
    ("rows 64x128", [40, 0, 71, 33] * 12, 504, "kn"),
    ("rows 128x64", [310, 0, 600, 290], 712, "kn"),
    ("rows 128x128", [120, 1, 140, 243] * 8, 504, "kn"),
    ("rows 128x128 in two stages", [310, 0, 600, 290] * 4, 440, "kn"),
    ("rows 128x256", [150, 0, 97, 128, 129] * 4, 2104, "kn"),
    ("ping-pong 256x256", [700, 0, 1, 900, 511], 5400, "kn"),
]
ROWS_16_UNALIGNED = [
    ("unaligned rows 32x64", [5, 0, 17, 3], 136, "kn"),
    ("unaligned rows 64x128", [40, 0, 71, 33] * 12, 1104, "kn"),
    ("unaligned rows 128x128", [128, 1, 140, 243] * 8, 504, "kn"),
]
ROWS_F32 = [
    ("fp32 stream 16x32", [5, 0, 17, 3], 136, "kn"),
    ("fp32 stream 32x64", [40, 0, 71, 33], 136, "kn"),
    ("fp32 stream 32x32", [130, 0, 60], 136, "kn"),
]
ROWS_F32_ALIGNED = [
    ("fp32 rows 64x64", [128, 1, 140, 243] * 4, 1104, "kn"),
    ("fp32 rows 64x128", [700, 0, 1, 900, 511], 5400, "kn"),
]
ROWS_F32_UNALIGNED = [("fp32 64x64 in two stages", [128, 1, 140, 243] * 4, 1104, "kn")]

# kernel: groups' k, M, N
K_16 = [
    ("k 64x64", [65, 0, 1, 130, 64], 136, 200),
    ("k 128x128", [33, 0, 64, 65] * 8, 504, 248),
    ("k 128x128 in two stages", [65, 0, 1, 130, 64, 200, 7, 128], 1000, 1000),
    ("ping-pong 256x256", [65, 0, 1, 130, 64], 1096, 2104),
]
K_16_UNALIGNED = [
    ("unaligned k 64x64", [65, 0, 1, 130, 64], 136, 200),
    ("unaligned k 128x128", [65, 0, 1, 130, 64, 200, 7, 128], 1000, 1000),
]
K_F32 = [
    ("fp32 64x64 in two stages", [65, 0, 1, 130, 64], 136, 200),
    ("fp32 k 128x128", [65, 0, 33], 2104, 2600),
]

# kernel: rows, N
LORA_16 = [
    ("stream 16x16", 12, 200, "k"),
    ("stream 16x32", 24, 200, "k"),
    ("16x32", 24, 200, "n"),
    ("32x32", 90, 200, "kn"),
    ("shared 32x32", 130, 200, "kn"),
    ("shared 64x64", 300, 520, "kn"),
    ("shared 64x64 in four stages", 515, 2056, "kn"),
    ("shared 128x128", 1500, 1504, "kn"),
    ("shared ping-pong 256x256", 2312, 2568, "kn"),
]
LORA_16_UNALIGNED = [
    ("unaligned 32x32", 130, 200, "kn"),
    ("unaligned 64x64", 300, 520, "kn"),
    ("unaligned 128x128", 1500, 1504, "kn"),
    ("unaligned 256x128", 4008, 2600, "kn"),
]
LORA_F32 = [
    ("stream 16x16", 12, 200, "kn"),
    ("stream 16x32", 24, 200, "kn"),
    ("stream 32x32", 90, 200, "kn"),
]
LORA_F32_ALIGNED = [("fp32 64x64", 1000, 1504, "kn"), ("fp32 64x128", 2312, 2568, "kn")]
LORA_F32_UNALIGNED = [("unaligned fp32 64x64", 1000, 1504, "kn")]

# What the tests of infinities and of v's last bits run, by type and padding.
LORA_VALUES = {
    (False, 0): {(1, 72): "stream 16x16", (24, 72): "stream 16x32", (48, 136): "32x32", (140, 136): "shared 32x32",
                 (300, 520): "shared 64x64", (515, 2056): "shared 64x64 in four stages",
                 (1500, 1504): "shared 128x128", (2312, 2568): "shared ping-pong 256x256"},
    (False, 1): {(1, 72): "unaligned 32x32", (300, 520): "unaligned 64x64", (515, 2056): "unaligned 64x64",
                 (1500, 1504): "unaligned 128x128", (4008, 2600): "unaligned 256x128"},
}


def grouped(f32, pad):
    """(kernel, groups' rows, N, orders of B) and (kernel, groups' k, M, N) of a type and padding."""
    if f32:
        return ROWS_F32 + (ROWS_F32_UNALIGNED if pad else ROWS_F32_ALIGNED), K_F32
    return (ROWS_16_UNALIGNED, K_16_UNALIGNED) if pad else (ROWS_16, K_16)


def lora(f32, pad):
    """(kernel, rows, N, orders of B) of a type and padding."""
    if f32:
        return LORA_F32 + (LORA_F32_UNALIGNED if pad else LORA_F32_ALIGNED)
    return LORA_16_UNALIGNED if pad else LORA_16
