"""Sizes that reach each kernel of expert_product_mxfp4, by the form that
csrc/experts_rules.hpp gives them.  The GPU tests run these sizes; test_experts_rules_host.py holds
them to the rules, so that a change of a rule cannot take a kernel out of the tests unseen."""

# (rows of the buffer, E, N) by the rows of a tile
PRODUCT = {
    32: [(20, 3, 304), (171, 3, 304), (90, 1, 272)],
    64: [(64, 1, 9472), (200, 5, 2592), (41, 24, 1072)],
    128: [(300, 2, 13456), (900, 12, 2832), (460, 5, 6416)],
    256: [(513, 1, 19808), (700, 3, 13600), (1800, 6, 5136)],
}
