"""Shapes (t, n, k) of the 8-bit linear and the gated half, one for every form that the plan can choose.

Tiles: (gated, float32 output, tile, K split or not).  Streams: (gated, waves, token tiles).  Widths k are whole 16-byte
pieces but no whole blocks, so that codes are read in place and end inside a block; t and n are odd.
"""
TILES = {
    (0, 0, 0, 0): (1176, 9231, 272), (0, 0, 0, 1): (4143, 149, 16976),
    (0, 0, 1, 0): (2440, 3191, 272), (0, 0, 1, 1): (141, 5609, 6176),
    (0, 0, 2, 0): (3589, 1109, 272), (0, 0, 2, 1): (129, 5773, 5456),
    (0, 0, 3, 0): (1157, 1717, 272), (0, 0, 3, 1): (198, 1351, 6928),
    (0, 0, 4, 0): (774, 1219, 272), (0, 0, 4, 1): (67, 1349, 2784),
    (0, 0, 5, 0): (798, 2333, 272), (0, 0, 5, 1): (692, 207, 4144),
    (0, 0, 6, 0): (65, 17, 272), (0, 0, 6, 1): (68, 19, 944),
    (1, 0, 0, 0): (1540, 3591, 272), (1, 0, 0, 1): (428, 1401, 13840),
    (1, 0, 1, 0): (2976, 1309, 272), (1, 0, 1, 1): (132, 2721, 6736),
    (1, 0, 2, 0): (1157, 1717, 272), (1, 0, 2, 1): (129, 1355, 10848),
    (1, 0, 3, 0): (783, 1285, 272), (1, 0, 3, 1): (69, 1367, 5920),
    (1, 0, 4, 0): (388, 1171, 272), (1, 0, 4, 1): (67, 691, 2576),
    (1, 0, 5, 0): (518, 1661, 272), (1, 0, 5, 1): (267, 389, 3488),
    (1, 0, 6, 0): (65, 17, 272), (1, 0, 6, 1): (68, 19, 944),
}
# float32 outputs leave out the three largest tiles and choose alike among the others
TILES.update({(g, 1, tile, split): shape for (g, _, tile, split), shape in list(TILES.items()) if tile >= 3})

STREAMS = {(g, waves, tiles): shape for g in (0, 1)
           for (waves, tiles), shape in {(16, 1): (11, 49, 8224), (8, 1): (13, 49, 1040), (8, 2): (17, 17, 1104),
                                         (8, 4): (33, 19, 1056)}.items()}
