"""Sizes that several test files of the feed-forward operators share."""

# (4-bit, gated, tokens, features, columns) of forward products that the tile kernel
# takes in more than two rounds of tiles, over many more K blocks than it has stages.
MANY_ROUNDS = [(False, True, 3003, 2056, 1544), (False, True, 2900, 2213, 776), (True, False, 3001, 4099, 2050),
               (True, False, 4500, 2561, 3334), (True, True, 2000, 2600, 3300), (True, True, 3333, 1411, 2050)]
