"""Sizes that reach each kernel of expert_product_mxfp4 and experts_decode, by the form that
csrc/experts_rules.hpp gives them.  The GPU tests run these sizes; test_experts_rules_host.py holds
them to the rules, so that a change of a rule cannot take a kernel out of the tests unseen."""

# (rows of the buffer, E, N) by the rows of a tile
PRODUCT = {
    32: [(20, 3, 304), (171, 3, 304), (90, 1, 272)],
    64: [(64, 1, 9472), (200, 5, 2592), (41, 24, 1072)],
    128: [(300, 2, 13456), (900, 12, 2832), (460, 5, 6416)],
    256: [(513, 1, 19808), (700, 3, 13600), (1800, 6, 5136)],
}

# (T, H, I, E, K) and the forms (entries at a time, elements of a stage, waves, split, parts of h as
# columns) of the two products with a bf16 result; with an f32 one packed columns hold 5 entries.
# Where a form takes many weight rows there is a size whose items are more than fit the card at once,
# with more than one group of stages each, and one with rows of whole cache lines.
BF16 = {
    (1, 72, 136, 5, 3): ((16, 64, 4, True, False), (16, 64, 2, False, False)),
    (1, 128, 192, 5, 3): ((16, 64, 4, True, False), (16, 64, 2, False, False)),
    (70, 712, 2600, 11, 1): ((16, 64, 2, False, False), (16, 64, 2, False, False)),
    (70, 5800, 808, 11, 1): ((16, 64, 2, False, False), (16, 64, 2, False, False)),
    (70, 704, 832, 11, 1): ((16, 64, 2, False, False), (16, 64, 2, False, False)),
    (30, 1160, 840, 56, 4): ((16, 64, 4, False, False), (16, 64, 4, False, False)),
    (30, 1152, 896, 60, 4): ((16, 64, 4, False, False), (16, 64, 4, False, False)),
    (40, 600, 3304, 9, 2): ((32, 64, 2, False, False), (32, 64, 2, False, False)),
    (40, 7160, 936, 9, 2): ((32, 64, 2, False, False), (32, 64, 2, False, False)),
    (40, 576, 960, 9, 2): ((32, 64, 2, False, False), (32, 64, 2, False, False)),
    (128, 1096, 1064, 60, 8): ((32, 64, 4, False, False), (32, 64, 4, False, False)),
    (128, 1088, 1088, 60, 8): ((32, 64, 4, False, False), (32, 64, 4, False, False)),
}
MXFP4 = {
    (1, 96, 160, 5, 3): ((16, 128, 4, True, False), (8, 128, 2, False, True)),
    (1, 96, 800, 5, 3): ((16, 128, 4, True, False), (8, 256, 2, False, True)),
    (1, 256, 1024, 5, 3): ((16, 128, 4, True, False), (8, 256, 2, False, True)),
    (33, 160, 64, 2, 2): ((16, 128, 4, True, False), (16, 128, 2, False, False)),
    (50, 672, 640, 30, 2): ((16, 128, 2, False, False), (8, 128, 2, False, True)),
    (50, 2144, 1120, 30, 2): ((16, 256, 4, False, False), (8, 256, 2, False, True)),
    (50, 1280, 1024, 30, 2): ((16, 256, 2, False, False), (8, 256, 2, False, True)),
    (40, 2080, 736, 96, 4): ((16, 256, 4, False, False), (8, 128, 4, False, True)),
    (40, 2080, 1312, 96, 4): ((16, 256, 4, False, False), (8, 256, 4, False, True)),
    (40, 2048, 1280, 96, 4): ((16, 256, 4, False, False), (8, 256, 4, False, True)),
    (60, 608, 1376, 60, 2): ((16, 128, 4, False, False), (8, 256, 2, False, True)),
    (140, 1824, 1248, 25, 2): ((16, 256, 2, False, False), (16, 128, 2, False, False)),
    (120, 2144, 1184, 64, 4): ((16, 256, 4, False, False), (16, 128, 4, False, False)),
    (128, 2208, 1120, 30, 8): ((32, 128, 4, False, False), (32, 128, 4, False, False)),
    (700, 4128, 2080, 16, 1): ((32, 128, 4, False, False), (32, 128, 4, False, False)),
}
