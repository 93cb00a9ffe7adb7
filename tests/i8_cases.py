"""Shapes that reach each form of the 8-bit linear's tensor-core kernels on a GPU of 148 SMs (csrc/i8_plan.h decides;
tests/test_i8_plan.py holds these shapes to it)."""

# M, N, K, columns per tile, whether those are tokens (swap): every width, with a K that wraps the ring of loads, an
# odd edge, and one tile a CTA pair or several
TILES = [
    (8904, 35, 1648, 32, False), (8595, 67, 1584, 64, False), (280, 3249, 1712, 96, False), (310, 4455, 1616, 128, False),
    (809, 2573, 1552, 160, False), (379, 6511, 1552, 192, False), (893, 3611, 1568, 224, False), (1824, 2053, 1648, 256, False),
    (1292, 4715, 656, 128, False), (593, 11405, 672, 160, False), (348, 19087, 672, 192, False), (590, 16331, 672, 224, False),
    (1462, 9417, 656, 256, False),
    (260, 7149, 144, 64, True), (281, 5755, 1936, 96, True), (578, 3379, 1568, 128, True), (516, 4295, 1552, 160, True),
    (325, 9381, 1552, 192, True), (786, 4315, 1568, 224, True), (337, 21900, 688, 128, True), (262, 19231, 704, 160, True),
    (533, 15211, 656, 192, True), (833, 12615, 656, 224, True),
]
# M, N, K, blocks of tokens, blocks a group: several groups, the last one short
GROUPS = [(1280, 600, 65536, 5, 2), (2500, 3000, 29584, 10, 4), (1044, 1834, 29584, 9, 5)]
# M, N, K, parts of K: 129 to 256 tokens that take the split-K kernel instead of tiles, every split that the rule takes
# for them on 148 SMs
SPLITS = [
    (145, 5098, 7952, 3), (240, 4500, 28672, 3), (129, 37, 5936, 4), (255, 3900, 9008, 4), (256, 1900, 10000, 4),
    (136, 32, 7024, 5), (201, 2600, 9008, 5), (129, 33, 8208, 6), (131, 36, 9872, 7), (199, 1900, 20000, 7),
    (131, 33, 11680, 8), (160, 1500, 131056, 8),
]
# clusters of 2 to 8 CTAs that 148 SMs held, at one CTA per SM and at two
HELD = {1: (74, 45, 33, 26, 22, 15, 15), 2: (148, 93, 71, 56, 45, 37, 33)}
