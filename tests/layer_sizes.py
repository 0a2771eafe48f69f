"""Sizes (tokens, width, hidden) of the feed-forward block that between them run
each of its five products with both tiles (128 and 256) and each way of its K:
no tile's split, all tiles' split, and whole rounds of tiles beside a split rest.
``test_layer_cover.py`` holds the list to that; the numbers of tokens, widths and
hidden values are no multiples of a tile, so each has ragged ends."""

TILES = [(62, 72, 72), (66, 1168, 2200), (22138, 456, 368), (644, 2776, 6072), (33090, 408, 712), (7181, 1128, 1816),
         (930, 2664, 2064), (65688, 1272, 136), (1999, 1600, 4264)]
