"""Sizes (rows, columns of the result, K) for which each kernel of the gated and the 8-bit integer products is the one
that is chosen, with its name as tests/c_client/ffn_launch_plan.cpp writes it.  tests/test_ffn_launch_plan.py holds the
names to the rule; tests/test_gpu_ffn_kernels.py runs the sizes.

Integers have odd sizes and a K that ends inside a group; teams of waves get every remainder of groups."""

INT8 = [
    (3, 3001, 1101, "stream 1x1x16"), (3, 5001, 1101, "stream 1x1x8"), (9, 6201, 1101, "stream 1x2x8"),
    (30, 3001, 1101, "stream 2x1x16"), (30, 5001, 1101, "stream 2x1x8"), (30, 6201, 1101, "stream 2x2x8"),
    (40, 5801, 1101, "stream 4x1x8"), (40, 6201, 1101, "stream 4x2x8"),
    (333, 1999, 1537, "tile 64x64x2"), (333, 999, 1250, "tile 64x64x2"),
    (200, 1000, 2433, "tile 64x64x4"), (200, 1000, 2600, "tile 64x64x4"), (200, 1000, 2700, "tile 64x64x4"),
    (200, 1000, 2817, "tile 64x64x4"),
    (777, 5001, 1030, "tile 128x128x1"), (500, 7000, 2300, "tile 128x128x2"), (500, 7000, 2431, "tile 128x128x2"),
    (2040, 8150, 1101, "tile 256x256x1"),
    (2040, 17341, 700, "tile 256x256x1 + 64x64x2"), (1837, 8310, 2494, "tile 256x256x1 + 64x64x4"),
    (9232, 10936, 153, "tile 256x256x1 + 128x128x1"), (8223, 2101, 1156, "tile 256x256x1 + 128x128x2"),
]

INT8_GATED = [
    (1, 2041, 1101, "stream half 1x1x16"), (29, 1408, 1101, "stream half 2x1x16"),
    (3, 2555, 1101, "stream 1x1x16"), (9, 6141, 1101, "stream 1x1x8"), (30, 3201, 1101, "stream 2x1x16"),
    (20, 6001, 1101, "stream 2x1x8"), (45, 3201, 1101, "stream 4x1x8"),
    (333, 999, 1537, "tile 64x64x2"), (333, 499, 1250, "tile 64x64x2"),
    (200, 513, 2433, "tile 64x64x4"), (200, 513, 2600, "tile 64x64x4"), (200, 513, 2700, "tile 64x64x4"),
    (200, 513, 2900, "tile 64x64x4"),
    (777, 2501, 1030, "tile 128x128x1"), (500, 3501, 2300, "tile 128x128x2"), (500, 3501, 2431, "tile 128x128x2"),
    (2040, 4075, 1101, "tile 256x256x1"),
    (2040, 8670, 700, "tile 256x256x1 + 64x64x2"), (3588, 2246, 2446, "tile 256x256x1 + 64x64x4"),
    (732, 12875, 850, "tile 256x256x1 + 128x128x1"), (1351, 6589, 1386, "tile 256x256x1 + 128x128x2"),
]

FP8_GATED = [
    (1, 2048, 1152, "stream half 1x1x16"), (29, 1408, 1152, "stream half 2x1x16"),
    (3, 2560, 1152, "stream 1x1x16"), (9, 6144, 1152, "stream 1x1x8"), (30, 3200, 1152, "stream 2x1x16"),
    (20, 6144, 1152, "stream 2x1x8"), (45, 3200, 1152, "stream 4x1x8"),
    (333, 1024, 1664, "tile 64x64x2"), (333, 512, 1280, "tile 64x64x2"),
    (200, 512, 2560, "tile 64x64x4"), (200, 512, 2688, "tile 64x64x4"), (200, 512, 2816, "tile 64x64x4"),
    (200, 512, 2944, "tile 64x64x4"),
    (1511, 2048, 1152, "tile 128x128x1"), (500, 3584, 2304, "tile 128x128x2"), (500, 3584, 2432, "tile 128x128x2"),
    (2040, 4096, 1152, "tile 256x256x1"),
    (2040, 8704, 640, "tile 256x256x1 + 64x64x2"), (1148, 6912, 2560, "tile 256x256x1 + 64x64x4"),
    (1713, 11520, 512, "tile 256x256x1 + 128x128x1"), (4713, 3712, 768, "tile 256x256x1 + 128x128x2"),
]
